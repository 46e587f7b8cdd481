"""What the int8 row products and the row sampler are measured on.

``listed()`` and ``draw()`` give cases, ``prepare()`` makes one case's inputs, ``run()`` passes once through
an operator: in its plain form (elementary torch operations), or, with ``own`` set, through the library's
entry points.  ``exact()`` is the operators' definition in 64 bits.

Three kinds of case:
  linear   activations [m, k] quantised row by row to int8, times int8 weights [n, k] with a scale per row
  matmul   the product alone, of activations that are int8 with a scale per row already
  sample   one token drawn for each row of logits [r, v] with temperature, top-k, top-p and min-p
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    return [
        # One token through a small square projection: the smallest call, all latency.
        dict(name="linear 1x1024x1024 bf16", op="linear", m=1, n=1024, k=1024, dtype="bf16", out="bf16", bias=False),
        # One token against an output head of 100k rows of depth 768: a read of the weights.
        dict(name="linear 1x100000x768 bf16", op="linear", m=1, n=100000, k=768, dtype="bf16", out="fp32", bias=False),
        # A batch of 32 decoding requests through a large projection.
        dict(name="linear 32x16384x4096 bf16", op="linear", m=32, n=16384, k=4096, dtype="bf16", out="bf16", bias=False),
        # A short ragged prompt through a projection with odd sizes and a bias.
        dict(name="linear 77x1001x777 fp16", op="linear", m=77, n=1001, k=777, dtype="fp16", out="fp16", bias=True),
        # A prompt of 2048 tokens through a square projection.
        dict(name="linear 2048x4096x4096 bf16", op="linear", m=2048, n=4096, k=4096, dtype="bf16", out="bf16", bias=False),
        # Scores in fp32 of 500 quantised rows against a resident corpus of 50k rows.
        dict(name="matmul 500x50000x768 fp32", op="matmul", m=500, n=50000, k=768, dtype="fp32", out="fp32", bias=False),
        # The largest product: a batch of long prompts through a large projection.
        dict(name="matmul 8192x8192x8192 bf16", op="matmul", m=8192, n=8192, k=8192, dtype="bf16", out="bf16", bias=False),
        # One request, a small vocabulary, the usual settings.
        dict(name="sample 1x32000 fp32 k+p", op="sample", r=1, v=32000, dtype="fp32", mode="kp", masked=0.0),
        # One request, a large vocabulary, top-p alone: every weight counts.
        dict(name="sample 1x131072 bf16 p", op="sample", r=1, v=131072, dtype="bf16", mode="p", masked=0.0),
        # A served batch: each request with its own settings, banned tokens, one row with nothing left.
        dict(name="sample 64x50001 fp16 mixed", op="sample", r=64, v=50001, dtype="fp16", mode="mixed", masked=0.1),
        # A large batch over a large vocabulary, top-p with min-p.
        dict(name="sample 256x131072 bf16 p+m", op="sample", r=256, v=131072, dtype="bf16", mode="pm", masked=0.0),
        # A very large batch of fp32 scores, each row with its own settings.
        dict(name="sample 512x100000 fp32 mixed", op="sample", r=512, v=100000, dtype="fp32", mode="mixed", masked=0.02),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["fp32", "bf16", "fp16"])
    if rng.random() < 0.5:
        while True:
            m, n, k = _log_int(rng, 1, 8192), _log_int(rng, 64, 131072), _log_int(rng, 64, 8192)
            if rng.random() < 0.5:  # half of the cases have depths as models have them
                k = max(64, k // 64 * 64)
            if m * n * k <= 8192 ** 3 and m * n <= 8192 ** 2:
                break
        op = rng.choice(["linear", "linear", "matmul"])
        return dict(op=op, m=m, n=n, k=k, dtype=dtype, out=rng.choice(["fp32", "bf16", "fp16"]), bias=rng.random() < 0.3)
    while True:
        r, v = _log_int(rng, 1, 512), _log_int(rng, 16, 262144)
        if r * v <= 512 * 100000:
            break
    return dict(op="sample", r=r, v=v, dtype=dtype, mode=rng.choice(["kp", "p", "pm", "m", "k", "t", "mixed"]),
                masked=rng.choice([0.0, 0.0, 0.05, 0.5]))


# -- inputs ------------------------------------------------------------------


def _rows_to_int8(x):
    """The definition, plainly: a scale of max/127 per row, whole numbers nearest to the exact quotient."""
    x = x.float()
    amax = x.abs().amax(1)
    scale = amax / torch.full_like(amax, 127.0)
    scale = torch.where(scale >= torch.finfo(torch.float32).tiny, scale, torch.zeros_like(scale))
    scale = torch.where(torch.isfinite(amax), scale, torch.full_like(scale, float("nan")))
    fine = scale > 0
    # in 64 bits: a quotient next to a half must not be rounded to it first
    q = torch.round(x.double() / torch.where(fine, scale, torch.ones_like(scale)).double()[:, None])
    q = torch.where(fine[:, None], q, torch.zeros_like(q)).to(torch.int8)
    return q, scale


def _weights(n, k, g):
    """int8 rows as a program keeps them: row stride a multiple of 16, made block by block."""
    w = torch.zeros(n, (k + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    scale = torch.empty(n, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 25) // k)
    for i in range(0, n, step):
        rows = torch.randn(min(step, n - i), k, device="cuda", generator=g) * 0.02
        q, s = _rows_to_int8(rows)
        w[i:i + step, :k] = q
        scale[i:i + step] = s
    return w[:, :k], scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if case["op"] != "sample":
        m, n, k = case["m"], case["n"], case["k"]
        x = torch.randn(m, k, device="cuda", generator=g)
        # some channels carry much larger activations than the rest
        x = x * (1.0 + 9.0 * (torch.rand(1, k, device="cuda", generator=g) < 0.01))
        w, w_scale = _weights(n, k, g)
        bias = torch.randn(n, device="cuda", generator=g) if case["bias"] else None
        state = dict(case=case, w=w, w_scale=w_scale, bias=bias, out=_TYPES[case["out"]])
        if case["op"] == "linear":
            state["x"] = x.to(_TYPES[case["dtype"]])
        else:
            a = torch.zeros(m, (k + 15) // 16 * 16, dtype=torch.int8, device="cuda")
            q, a_scale = _rows_to_int8(x.to(_TYPES[case["dtype"]]))
            a[:, :k] = q
            state.update(a=a[:, :k], a_scale=a_scale)
        return state
    r, v = case["r"], case["v"]
    # logits of a language model: a wide bulk and, in each row, a few dozen tokens that stand out
    x = torch.randn(r, v, device="cuda", generator=g) * 2.0
    hot = torch.rand(r, v, device="cuda", generator=g) < min(1.0, 48 / v)
    x += hot * (torch.rand(r, v, device="cuda", generator=g) * 8.0 + 2.0)
    x = x.to(_TYPES[case["dtype"]])
    if case["masked"]:
        x.masked_fill_(torch.rand(r, v, device="cuda", generator=g) < case["masked"], float("-inf"))
    mode = case["mode"]
    settings = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    if mode == "kp":
        settings.update(temperature=0.8, top_k=50, top_p=0.9)
    elif mode == "k":
        settings.update(temperature=0.7, top_k=200)
    elif mode == "p":
        settings.update(temperature=1.0, top_p=0.95)
    elif mode == "pm":
        settings.update(temperature=0.9, top_p=0.98, min_p=0.002)
    elif mode == "m":
        settings.update(temperature=1.2, min_p=0.05)
    elif mode == "mixed":
        # each request has its own settings; some are greedy, some leave a filter out
        def pick(values, dtype):
            values = torch.tensor(values, dtype=dtype, device="cuda")
            return values[torch.randint(0, len(values), (r,), device="cuda", generator=g)]
        settings = dict(temperature=pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3], torch.float32),
                        top_k=pick([0, 0, 20, 50, 100, 1000], torch.int32),
                        top_p=pick([1.0, 0.8, 0.9, 0.95, 0.99], torch.float32),
                        min_p=pick([0.0, 0.0, 0.01, 0.05], torch.float32))
        if r > 8:
            x[r // 2] = float("-inf")  # a request whose mask leaves nothing
    return dict(case=case, x=x, u=torch.rand(r, device="cuda", generator=g), settings=settings)


# -- the plain forms -----------------------------------------------------------


def _product_plain(a, a_scale, w, w_scale, bias, out):
    y = (a.float() @ w.float().t()) * a_scale[:, None] * w_scale[None, :]
    if bias is not None:
        y = y + bias
    return y.to(out)


def _column(value, like, dtype):
    if isinstance(value, torch.Tensor):
        return value.to(dtype)[:, None]
    # a plain number acts as the fp32 number that the library takes
    return torch.full((like.shape[0], 1), np.float32(value).item() if dtype == torch.float64 else value,
                      dtype=dtype, device=like.device)


def _sample_plain(x, u, temperature, top_k, top_p, min_p):
    """Sorted order, running sums and the draw in 64 bits: a token is decided by which side of a border its sum lies on."""
    v = x.shape[1]
    x = x.float()
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x) + 0.0
    t, k = _column(temperature, x, torch.float64), _column(top_k, x, torch.int64)
    p, least = _column(top_p, x, torch.float64), _column(min_p, x, torch.float64)
    greedy = ~(t > 0)
    top = x.amax(1, keepdim=True)
    empty = top == float("-inf")
    w = torch.exp((x.double() - top.double()) / torch.where(greedy, torch.ones_like(t), t))
    w = torch.where(x == top, torch.ones_like(w), w)
    w = torch.where(empty, torch.zeros_like(w), w)
    _, order = torch.sort(x, dim=1, descending=True, stable=True)
    sw = torch.gather(w, 1, order)
    rank = torch.arange(v, device=x.device)[None, :]
    keep = rank < torch.where(k > 0, k, torch.full_like(k, v))
    run_k = torch.cumsum(torch.where(keep, sw, torch.zeros_like(sw)), 1)
    before = torch.cat([torch.zeros_like(run_k[:, :1]), run_k[:, :-1]], 1)
    keep = keep & ((p >= 1) | (before < p * run_k[:, -1:])) & (sw >= least)
    keep = torch.where(greedy, rank == 0, keep | (rank == 0))
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    wk = torch.where(kept, w, torch.zeros_like(w))
    run = torch.cumsum(wk, 1)
    total = run[:, -1:]
    token = torch.minimum((run <= u.double()[:, None] * total).sum(1), (run < total).sum(1)).clamp(max=v - 1)
    prob = torch.gather(wk, 1, token[:, None])[:, 0] / total[:, 0]
    gone = empty[:, 0]
    return (torch.where(gone, torch.full_like(token, -1), token).to(torch.int32),
            torch.where(gone, torch.zeros_like(prob), prob).float())


def run(state):
    op = state["case"]["op"]
    if own:
        import top_search_resident_amd as rt
        if op == "linear":
            return rt.linear_int8(state["x"], state["w"], state["w_scale"], bias=state["bias"], out_dtype=state["out"])
        if op == "matmul":
            return rt.matmul_int8(state["a"], state["a_scale"], state["w"], state["w_scale"], bias=state["bias"],
                                  out_dtype=state["out"])
        return rt.sample_rows(state["x"], state["u"], **state["settings"])
    if op == "linear":
        q, scale = _rows_to_int8(state["x"])
        return _product_plain(q, scale, state["w"], state["w_scale"], state["bias"], state["out"])
    if op == "matmul":
        return _product_plain(state["a"], state["a_scale"], state["w"], state["w_scale"], state["bias"], state["out"])
    return _sample_plain(state["x"], state["u"], **state["settings"])


def work(case):
    if case["op"] == "sample":
        # each logit once, the settings and the number per row, token and probability out; a subtraction,
        # an exponential and a sum for each logit
        n = case["r"] * case["v"]
        return {"bytes": n * _SIZE[case["dtype"]] + case["r"] * 12, "flops": 3 * n}
    m, n, k = case["m"], case["n"], case["k"]
    act = m * k * _SIZE[case["dtype"]] if case["op"] == "linear" else m * k + 4 * m
    return {"bytes": act + n * k + 4 * n + (4 * n if case["bias"] else 0) + m * n * _SIZE[case["out"]],
            "flops": 2 * m * n * k}


# -- the definitions in 64 bits ------------------------------------------------


def _exact_rows(x):
    """int8 rows as 64-bit whole values and their scales, from the quotient's remainder."""
    x = x.double()
    amax = x.abs().max(dim=1).values
    scale = (amax / 127).float().double()
    scale[scale < 2.0 ** -126] = 0
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    q = torch.floor(x / safe)
    rest = x - q * safe - safe / 2
    q = q + ((rest > 0) | ((rest == 0) & (q % 2 == 1))).double()
    return torch.where(scale[:, None] > 0, q, torch.zeros_like(q)), scale


def _exact_draw(x, u, t, k, p, least):
    """One row on the host; x is a float64 array."""
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1, 0.0
    if not t > 0:
        return int(np.argmax(x)), 1.0
    live = np.flatnonzero(x > -np.inf)  # ascending: a stable sort keeps ties in the order of their index
    order = live[np.argsort(-x[live], kind="stable")]
    with np.errstate(under="ignore", invalid="ignore"):
        w = np.where(x[order] == top, 1.0, np.exp((x[order] - top) / t))
    if 0 < k < len(order):
        order, w = order[:k], w[:k]
    last = len(order)
    if p < 1:
        last = int(np.searchsorted(np.cumsum(w), p * w.sum(), side="left")) + 1
    last = max(1, min(last, int(np.count_nonzero(w >= least))))
    order, w = order[:last], w[:last]
    by_index = np.argsort(order)
    order, w = order[by_index], w[by_index]
    run = np.cumsum(w)
    at = min(int(np.searchsorted(run, u * run[-1], side="right")), int(np.searchsorted(run, run[-1], side="left")))
    return int(order[at]), float(w[at] / run[-1])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "sample":
        a, a_scale = _exact_rows(s["x"]) if case["op"] == "linear" else (s["a"].double(), s["a_scale"].double())
        w, w_scale = s["w"], s["w_scale"].double()
        y = torch.empty(case["m"], case["n"], dtype=torch.float64, device="cuda")
        for i in range(0, case["n"], 16384):
            y[:, i:i + 16384] = torch.mm(a, w[i:i + 16384].double().t().contiguous()) * w_scale[i:i + 16384]
        y *= a_scale[:, None]
        if s["bias"] is not None:
            y += s["bias"].double()
        return y
    r = case["r"]

    def column(value, dtype):
        if isinstance(value, torch.Tensor):
            return value.cpu().numpy().astype(dtype)
        return np.full(r, np.float32(value) if dtype == np.float64 else value, dtype)

    st = s["settings"]
    t, k = column(st["temperature"], np.float64), column(st["top_k"], np.int64)
    p, least = column(st["top_p"], np.float64), column(st["min_p"], np.float64)
    u = s["u"].cpu().numpy().astype(np.float64)
    token, prob = np.empty(r, np.int32), np.empty(r, np.float64)
    for i in range(r):
        token[i], prob[i] = _exact_draw(s["x"][i].double().cpu().numpy(), u[i], t[i], k[i], p[i], least[i])
    return token, prob
