"""Row sampling on the GPU against the plain 64-bit definition: every filter
and their combinations, one logit to long rows, ties, masks, infinities and
NaN, extreme settings, strides, streams and graphs.

The kernel's sums are off by at most what row_oracle.draw works out from the
unit of its weights; a row whose decisions all stay further than that from a
border must give the same token.  The rows here do (asserted)."""
import numpy as np
import pytest

import row_oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from top_search_resident_amd import ResidentTopKError, linear_int8, quantize_rows_int8, sample_rows  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
NAN, INF = float("nan"), float("inf")


def per_row(value, r):
    return value.cpu().numpy() if isinstance(value, torch.Tensor) else [value] * r


def check(x, u, exact_ties=False, **settings):
    """x, u on the CPU; runs the kernel and compares every row."""
    gpu = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in settings.items()}
    token, prob = sample_rows(x if x.is_cuda else x.cuda(), u.cuda(), **gpu)
    token, prob = token.cpu().numpy(), prob.cpu().numpy()
    r, v = x.shape
    rows = x.double().cpu().numpy()
    s = {k: per_row(settings.get(k, d), r) for k, d in
         (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))}
    for i in range(r):
        e, p, margin, error = row_oracle.draw(rows[i], u[i].item(), s["temperature"][i], int(s["top_k"][i]),
                                       s["top_p"][i], s["min_p"][i])
        if not exact_ties:
            assert margin > error, ("the test's own row sits on a border", i, margin, error)
        assert token[i] == e, (i, token[i], e, margin)
        # the sum's error and one rounding to fp32
        assert abs(prob[i] - p) <= p * (2.0 ** -24 + error) * 1.01 + 2.0 ** -149, (i, prob[i], p)
    return token, prob


def logits(r, v, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(r, v, generator=g) * spread).to(TYPES[dtype]), torch.rand(r, generator=g)


FILTERS = [dict(), dict(temperature=0.7), dict(top_k=5), dict(top_k=1000), dict(top_p=0.9), dict(top_p=0.3),
           dict(min_p=0.05), dict(top_k=40, top_p=0.8), dict(top_p=0.95, min_p=0.01), dict(top_k=3000, top_p=0.97),
           dict(temperature=1.5, top_k=300, top_p=0.9, min_p=0.002), dict(temperature=0.05, top_k=50, top_p=0.99)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("v", [1, 2, 63, 1000, 8193, 50001])
@pytest.mark.parametrize("f", range(len(FILTERS)))
def test_filters(dtype, v, f):
    x, u = logits(5, v, dtype, 100 * v + f)
    check(x, u, **FILTERS[f])


@pytest.mark.parametrize("dtype,v,r", [("bf16", 131072, 2), ("bf16", 131072, 20), ("fp32", 262145, 2), ("fp16", 1000003, 2),
                                       ("fp32", 700001, 17)])
@pytest.mark.parametrize("f", [0, 4, 6, 7, 8, 9, 10])
def test_long_rows(dtype, v, r, f):
    x, u = logits(r, v, dtype, v + f)
    check(x, u, **FILTERS[f])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("f", range(len(FILTERS)))
def test_many_rows(dtype, f):
    x, u = logits(270, 6007, dtype, 500 + f)
    check(x, u, **FILTERS[f])


def test_long_rows_of_every_kind_at_once():
    """Shared rows (several workgroups each): empty, one token, greedy, infinite, tied, masked and flat rows
    with settings of their own, in one call; then each with no filter, top-p, min-p and top-k for all."""
    r, v = 8, 150000
    g = torch.Generator().manual_seed(30)
    x = torch.randn(r, v, generator=g)
    x[0] = -INF
    x[1] = NAN
    x[1, 140001] = 0.5
    x[2, ::2] = -INF
    x[3, [7, 77777, 149999]] = INF
    x[4] = 2.0
    x[5] = torch.randint(-4, 5, (v,), generator=g).float()
    x[6] = torch.finfo(torch.float32).min
    x[6, 99999] = 1.0
    u = torch.rand(r, generator=g)
    check(x, u, exact_ties=True, temperature=torch.tensor([1.0, 1.0, 0.0, 1.0, 1.0, 0.9, 1.0, 2.0]),
          top_k=torch.tensor([0, 50, 0, 2, 30000, 0, 9, 5000], dtype=torch.int32),
          top_p=torch.tensor([0.9, 0.5, 1.0, 1.0, 1.0, 0.7, 0.9, 0.95]),
          min_p=torch.tensor([0.0, 0.1, 0.0, 0.0, 0.0, 0.0, 0.01, 0.0]))
    for s in (dict(), dict(top_p=0.9), dict(min_p=0.2), dict(top_k=10), dict(top_k=40000, top_p=0.5), dict(temperature=0.0)):
        check(x, u, exact_ties=True, **s)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("r,v", [(40, 3001), (9, 200001), (3, 300000), (300, 700), (290, 20011)])
def test_settings_of_each_row(dtype, r, v):
    x, u = logits(r, v, dtype, 77 + r)
    g = torch.Generator().manual_seed(8)

    def pick(values, dt):
        return torch.tensor(values, dtype=dt)[torch.randint(0, len(values), (r,), generator=g)]

    # bf16 and fp16 rows this long hold their largest logit more than once: top_p 0.5 and min_p 1 then
    # meet exact ties, which whole weights decide as the definition does
    check(x, u, exact_ties=True, temperature=pick([0.0, 0.5, 1.0, 2.0, -1.0], torch.float32),
          top_k=pick([0, 1, 2, 50, 2000, 5000, -3], torch.int32),
          top_p=pick([1.0, 0.5, 0.9, 0.0, 2.0], torch.float32), min_p=pick([0.0, 0.1, 0.001, 1.0], torch.float32))


@pytest.mark.parametrize("top_k", [1, 2, 3, 7, 2500, 4095, 4096])
def test_ties_keep_the_lower_index(top_k):
    """All logits equal, and two levels: whole weights make every border exact."""
    v = 4096
    x = torch.zeros(8, v)
    x[4:] = torch.where(torch.arange(v) % 3 == 0, 1.5, -40.0)
    u = torch.tensor([0.0, 0.25, 0.5, 0.999] * 2)
    token, prob = check(x, u, exact_ties=True, top_k=top_k)
    assert (token[:4] == [int(q * top_k) for q in u[:4].tolist()]).all()
    assert np.all(prob[:4] == np.float32(1.0 / top_k))


@pytest.mark.parametrize("top_p,kept", [(0.5, 2048), (0.25, 1024), (1.0, 4096), (0.125, 512)])
def test_flat_rows_split_exactly(top_p, kept):
    x = torch.full((3, 4096), -7.25)
    token, prob = check(x, torch.tensor([0.0, 0.5, 0.99]), exact_ties=True, top_p=top_p)
    assert np.all(prob == np.float32(1.0 / kept)) and token[1] == kept // 2


def test_ties_of_signed_zeros_and_many_equal_logits():
    x = torch.zeros(2, 20000)
    x[:, ::2] = -0.0
    x[1, 7] = 0.5
    check(x, torch.tensor([0.3, 0.7]), exact_ties=True, top_k=33)
    # bf16 logits with a few values each held by thousands: the border lies inside a tie
    g = torch.Generator().manual_seed(4)
    y = torch.randint(-4, 5, (6, 60000), generator=g).to(torch.bfloat16)
    for s in (dict(top_k=10), dict(top_k=9000), dict(top_p=0.7), dict(top_p=0.999), dict(top_k=20000, top_p=0.5),
              dict(min_p=0.1)):
        check(y, torch.rand(6, generator=g), **s)


def test_masked_infinite_and_nan_logits():
    v = 5000
    g = torch.Generator().manual_seed(6)
    x = torch.randn(12, v, generator=g) * 3
    x[0] = -INF                               # nothing left
    x[1] = NAN
    x[2, 1:] = -INF                           # one token left
    x[3, :-1] = NAN
    x[4, ::2] = -INF
    x[5, 1::2] = NAN
    x[6, 100] = INF                           # one infinite logit takes all
    x[7, [9, 4000, 77]] = INF                 # three share
    x[8] = torch.finfo(torch.float32).min     # masks of the lowest value
    x[9] = torch.finfo(torch.float32).min
    x[9, 123] = 4.0
    x[10] = torch.finfo(torch.float32).max
    x[11, :4990] = -INF
    u = torch.rand(12, generator=g)
    for s in (dict(), dict(top_k=20), dict(top_p=0.9), dict(min_p=0.1), dict(temperature=0.0), dict(top_k=4999),
              dict(temperature=0.3, top_k=30, top_p=0.5, min_p=0.01)):
        token, prob = check(x, u, exact_ties=True, **s)
        assert (token[:2] == -1).all() and (prob[:2] == 0).all()
        assert token[2] == 0 and token[3] == v - 1 and token[6] == 100 and token[9] == 123
        assert token[7] in (9, 77, 4000)


@pytest.mark.parametrize("s", [dict(temperature=1e-30), dict(temperature=1e-45), dict(temperature=1e30),
                               dict(temperature=INF, top_k=7), dict(temperature=NAN), dict(temperature=-1.0),
                               dict(top_p=1e-9), dict(top_p=0.0), dict(top_p=-1.0), dict(top_p=NAN), dict(top_p=7.0),
                               dict(min_p=1.0), dict(min_p=1.5), dict(min_p=NAN), dict(min_p=1e-40), dict(min_p=-1.0),
                               dict(top_k=2 ** 40), dict(top_k=-5)])
def test_extreme_settings(s):
    x, u = logits(4, 900, "fp32", 12)
    check(x, u, exact_ties=True, **s)


@pytest.mark.parametrize("r,v", [(4, 900), (30, 9000), (2, 270000), (300, 5000)])
@pytest.mark.parametrize("s", [dict(), dict(min_p=1.0), dict(min_p=0.5), dict(top_p=0.5), dict(top_k=600, min_p=1.0)])
def test_infinite_temperature_weighs_all_the_same(r, v, s):
    x, u = logits(r, v, "fp32", 41)
    x[:, 1::3] = -INF
    check(x, u, exact_ties=True, temperature=INF, **s)


@pytest.mark.parametrize("r,v,first", [(24, 100001, 0), (24, 100001, 33000), (300, 20001, 10240), (2, 270000, 8200),
                                       (2, 270000, 0)])
def test_random_number_one_behind_the_rounded_sums(r, v, first):
    """The finite logits lie at the start of one of the parts whose weights are summed on their own,
    with nothing behind them there: the sums' last unit still draws the last of them."""
    g = torch.Generator().manual_seed(v + first)
    x = torch.full((r, v), -INF)
    x[:, first + 10:first + 900] = torch.randn(r, 890, generator=g) * 2
    for s in (dict(), dict(temperature=1.3), dict(top_p=0.9999), dict(min_p=1e-6)):
        for u in (1.0, 3.0, 1.0 - 2.0 ** -24):
            out = torch.full((r,), -7, dtype=torch.int32, device="cuda")
            sample_rows(x.cuda(), torch.full((r,), u).cuda(), out_token=out, **s)
            assert (out >= first + 10).all() and (out < first + 900).all()
            if u >= 1:
                check(x, torch.full((r,), u), exact_ties=True, **s)


@pytest.mark.parametrize("r", [2, 20])
def test_weights_that_only_together_make_a_unit(r):
    """Ten tokens of three tenths of the smallest unit each: their part of the row weighs 3 units, none of
    them alone one."""
    v = 140000  # units of 2^-44 of the largest weight
    x = torch.full((r, v), -INF)
    x[:, 5] = 0.0
    x[:, 131500:131510] = float(np.log(0.3 * 2.0 ** -44))
    check(x, torch.ones(r), exact_ties=True)


def test_longest_row():
    """2^31 - 1 logits, by many workgroups and (infinite ones) by one."""
    v = 2 ** 31 - 1
    x = torch.full((1, v), -INF, dtype=torch.bfloat16, device="cuda")
    places = [5, 70001, 2 ** 30 + 3, v - 9, v - 1]
    values = torch.tensor([1.0, 3.0, 2.0, 0.0, 2.5]).to(torch.bfloat16)
    x[0, places] = values.cuda()
    for u in (0.0, 0.3, 0.9, 1.0):
        for s in (dict(), dict(top_k=3), dict(top_p=0.6), dict(min_p=0.3), dict(temperature=0.0)):
            token, prob = sample_rows(x, torch.tensor([u]).cuda(), **s)
            e, p, margin, _ = row_oracle.draw(values.double().numpy(), u, **s)
            assert margin > 1e-6  # 5 weights, each off by half of 2^-31 at most
            assert token.item() == places[e] and abs(prob.item() - p) <= p * 1e-6
    x[0, places[1:4]] = INF
    assert sample_rows(x, torch.tensor([0.5]).cuda())[0].item() == places[2]


def test_rows_far_apart_and_more_rows_than_a_launch():
    far = torch.empty(3, 2 ** 31 - 1, dtype=torch.bfloat16, device="cuda")[:, :700]
    x, u = logits(3, 700, "bf16", 43)
    far.copy_(x)
    check(far, u, top_k=40, top_p=0.9)
    r = (1 << 20) + 3
    x = torch.randn(r, 3, generator=torch.Generator().manual_seed(44)).cuda()
    token, prob = sample_rows(x, torch.zeros(r, device="cuda"), temperature=0.0)
    assert torch.equal(token.long(), x.argmax(1)) and (prob == 1).all()


def test_random_numbers_at_the_ends():
    x, _ = logits(6, 700, "fp32", 13)
    x[:, :5] = -INF
    x[:, -5:] = -INF
    u = torch.tensor([0.0, -1.0, NAN, 1.0, 2.0, 1.0 - 2.0 ** -24])
    token, _ = check(x, u, exact_ties=True)
    assert (token[:3] == 5).all() and (token[3:5] == 694).all()


def test_every_kept_token_can_be_drawn():
    """A sweep of u over one row gives each kept token its share of the sweep."""
    x = torch.tensor([[0.0, 3.0, 1.0, 2.5, -1.0, 2.0]]).repeat(1000, 1)
    u = (torch.arange(1000) + 0.5) / 1000
    token, prob = sample_rows(x.cuda(), u.cuda(), top_k=4)
    token, prob = token.cpu().numpy(), prob.cpu().numpy()
    assert set(token) == {1, 2, 3, 5}
    w = {1: 1.0, 3: np.exp(-0.5), 5: np.exp(-1.0), 2: np.exp(-2.0)}
    for i, q in w.items():
        share = q / sum(w.values())
        assert abs(np.mean(token == i) - share) <= 2e-3  # a border moves one of 1000 steps at each end
        assert np.all(np.abs(prob[token == i] - share) <= share * 2.0 ** -23)
    assert (np.diff(token) >= 0).all()  # index order


def test_strides_and_given_outputs():
    x, u = logits(9, 1111, "bf16", 15)
    store = torch.full((9, 1300), 50.0).to(torch.bfloat16)
    store[:, 3:3 + 1111] = x
    view = store.cuda()[::2, 3:3 + 1111]
    tok = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    prob = torch.empty(5, device="cuda")
    got = sample_rows(view, u[::2].contiguous().cuda(), top_k=30, out_token=tok, out_prob=prob)
    assert got[0] is tok and got[1] is prob
    check(view, u[::2].contiguous(), top_k=30)
    e, _ = sample_rows(x.cuda()[::2].contiguous(), u[::2].contiguous().cuda(), top_k=30)
    assert torch.equal(tok, e)


def test_empty_batch():
    t, p = sample_rows(torch.empty(0, 10, device="cuda"), torch.empty(0, device="cuda"))
    assert t.shape == (0,) and p.shape == (0,)


def test_streams_at_once_and_same_answer_each_time():
    x, u = logits(3, 200000, "fp32", 16)
    y, w = logits(70, 30000, "bf16", 17)
    jobs = [(x.cuda(), u.cuda(), dict(top_p=0.95)), (y.cuda(), w.cuda(), dict(top_k=50, top_p=0.9))]
    first = [sample_rows(a, b, **s) for a, b, s in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(i, sample_rows(*jobs[i][:2], **jobs[i][2], stream=streams[i])) for _ in range(5) for i in range(2)]
    torch.cuda.synchronize()
    for i, g in got:
        assert torch.equal(g[0], first[i][0]) and torch.equal(g[1], first[i][1])


@pytest.mark.parametrize("r,v", [(1, 32000), (1, 300000), (33, 5000)])
def test_captured_and_replayed(r, v):
    x, u = logits(r, v, "fp32", 18)
    x, u = x.cuda(), u.cuda()
    s = dict(temperature=0.9, top_k=100, top_p=0.9)
    sample_rows(x, u, **s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tok, prob = sample_rows(x, u, **s)
    for seed in range(4):
        nx, nu = logits(r, v, "fp32", 50 + seed)
        x.copy_(nx)
        u.copy_(nu)
        graph.replay()
        got = tok.clone(), prob.clone()
        eager = sample_rows(x, u, **s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])
        check(nx, nu, **s)


def test_head_product_then_draw():
    """Hidden states through an int8 output head, then one token each: the
    tokens are those the plain definitions give for the head's own logits."""
    g = torch.Generator().manual_seed(20)
    w, sw = quantize_rows_int8((torch.randn(5003, 768, generator=g) * 0.05).cuda())
    hidden = torch.randn(6, 768, generator=g).to(torch.bfloat16).cuda()
    scores = linear_int8(hidden, w, sw, out_dtype=torch.float32)
    q, s = row_oracle.quantize_rows(hidden.double().cpu().numpy())
    y, prod = row_oracle.product(q, s, w.cpu().numpy(), sw.cpu().numpy())
    assert (np.abs(scores.double().cpu().numpy() - y) <= 3.01 * 2.0 ** -24 * prod).all()
    check(scores, torch.rand(6, generator=g), temperature=0.8, top_k=50, top_p=0.9)


def test_rejects_bad_arguments():
    x = torch.zeros(4, 32, device="cuda")
    u = torch.zeros(4, device="cuda")
    for bad in (lambda: sample_rows(x.double(), u), lambda: sample_rows(x.t(), u), lambda: sample_rows(x.cpu(), u),
                lambda: sample_rows(x, u.cpu()), lambda: sample_rows(x, u.double()),
                lambda: sample_rows(x, u, top_k=torch.ones(4, device="cuda")),
                lambda: sample_rows(x[:1].expand(4, 32), u)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: sample_rows(x, u[:3]), lambda: sample_rows(x[0], u),
                lambda: sample_rows(x, u, temperature=torch.ones(5, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ResidentTopKError):
        sample_rows(torch.empty(4, 0, device="cuda"), u)
