"""Cases of the products whose weights are chosen per row: experts' layers
and low-rank adapters of many requests.

Each case names its kind:

  order     group_rows(): the rows of every expert, from the router's choices
  experts   gemm_grouped(): one product of an experts' layer
  train     gemm_grouped(), then gemm_grouped_backward()
  combine   combine_rows(): each token's experts added by their weights, and
            with `train` combine_rows_backward()
  adapters  gemm_adapters(): a shared projection and the low-rank term of
            each row's adapter

`run` takes the plain form below, or with `own` the framework's entry points.
The plain form pads the groups to the longest and uses library products in
float32; `exact` is the definition in float64, group by group.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
          "i32": torch.int32, "i64": torch.int64}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "i32": 4, "i64": 8}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a batch: the router's choices of 128 tokens
        dict(name="order_decode", kind="order", ids="i64", tokens=128, top=8, groups=64,
             skew=0.5, padded=0.0),
        # a large batch of prompts, a tenth of it padding
        dict(name="order_prompt", kind="order", ids="i32", tokens=65536, top=8, groups=256,
             skew=0.5, padded=0.1),
        # a single token's two experts: the weights of both are read once
        dict(name="experts_token", kind="experts", dtype="bf16", out="bf16", tokens=1, top=2,
             groups=8, k=4096, n=2048, skew=0.0),
        # a decoding batch over many small experts, a few rows each
        dict(name="experts_decode", kind="experts", dtype="f16", out="f16", tokens=64, top=4,
             groups=64, k=2048, n=1024, skew=0.5),
        # a prompt whose experts are few and large
        dict(name="experts_prompt", kind="experts", dtype="bf16", out="bf16", tokens=8192, top=2,
             groups=8, k=4096, n=2048, skew=0.3),
        # an odd batch over uneven experts, some of them with next to nothing; fp32 results
        dict(name="experts_uneven", kind="experts", dtype="f16", out="f32", tokens=1021, top=3,
             groups=32, k=1000, n=2048, skew=1.5),
        # fine-tuning on a few short samples
        dict(name="train_short", kind="train", dtype="f16", tokens=333, top=2, groups=16, k=512,
             n=1024, skew=0.5),
        # pretraining: forward and both gradients
        dict(name="train_packed", kind="train", dtype="bf16", tokens=4096, top=2, groups=8,
             k=2048, n=4096, skew=0.3),
        # a decoding step's outputs added up per token
        dict(name="combine_decode", kind="combine", dtype="bf16", tokens=64, top=4, n=4096,
             missing=0.0, train=False),
        # a training batch, forward and gradients, some choices dropped
        dict(name="combine_train", kind="combine", dtype="bf16", tokens=8191, top=2, n=4096,
             missing=0.05, train=True),
        # a decoding batch: a row per request, some of them without an adapter
        dict(name="adapters_decode", kind="adapters", dtype="bf16", out="bf16", rows=48,
             adapters=16, rank=16, k=4096, n=4096, plain=0.2, runs=False),
        # packed prompts of a few requests
        dict(name="adapters_prompt", kind="adapters", dtype="f16", out="f16", rows=5001,
             adapters=8, rank=64, k=4096, n=4096, plain=0.1, runs=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _log_eight(rng, lo, hi):
    """A multiple of eight, as the products' sizes are."""
    return 8 * _log_int(rng, lo // 8, hi // 8)


def draw(rng):
    kind = rng.choice(["order", "experts", "experts", "train", "combine", "adapters", "adapters"])
    if kind == "order":
        case = dict(kind=kind, ids=rng.choice(["i32", "i64"]), tokens=_log_int(rng, 1, 65536),
                    groups=_log_int(rng, 2, 256), skew=rng.uniform(0, 2),
                    padded=rng.choice([0.0, 0.0, 0.1, 0.6]))
        case["top"] = rng.randint(1, min(8, case["groups"]))
        return case
    case = dict(kind=kind, dtype=rng.choice(["bf16", "f16"]))
    if kind == "combine":
        case.update(tokens=_log_int(rng, 1, 8191), n=_log_eight(rng, 64, 4096),
                    missing=rng.choice([0.0, 0.1]), train=rng.random() < 0.5)
        most = max(1, 8191 * 2 // case["tokens"])
        case["top"] = rng.randint(1, min(8, most))
        return case
    case.update(k=_log_eight(rng, 64, 4096), n=_log_eight(rng, 64, 4096))
    if kind == "adapters":
        case.update(out=rng.choice([case["dtype"], case["dtype"], "f32"]),
                    rows=_log_int(rng, 1, 5001), adapters=_log_int(rng, 1, 64),
                    rank=rng.choice([8, 8, 16, 16, 24, 32, 64]), plain=rng.choice([0.0, 0.2]),
                    runs=rng.random() < 0.5)
        return case
    case.update(groups=_log_int(rng, 2, 64), skew=rng.uniform(0, 1.5),
                tokens=_log_int(rng, 1, 8192 if kind == "experts" else 4096))
    case["top"] = rng.randint(1, min(8, case["groups"]))
    if kind == "experts":
        case["out"] = rng.choice([case["dtype"], case["dtype"], "f32"])
    # no dearer than the listed ones
    while case["groups"] * case["n"] * case["k"] > 64 * 2048 * 1024:
        case["groups"] = max(2, case["groups"] // 2)
        case["top"] = min(case["top"], case["groups"])
        if case["groups"] == 2:
            break
    while case["top"] > 1 and case["tokens"] * case["top"] > (16384 if kind == "experts" else 8192):
        case["top"] -= 1
    return case


def _reached(groups, tokens, share):
    """Groups that `tokens` draws of `share` of them reach, about."""
    return groups * (1 - (1 - share) ** tokens)


def work(case):
    kind = case["kind"]
    if kind == "order":
        n = case["tokens"] * case["top"]
        return {"bytes": n * (SIZE[case["ids"]] + 8) + 4 * (case["groups"] + 1), "flops": 2 * n}
    e = SIZE[case["dtype"]]
    if kind == "combine":
        t, m, n = case["tokens"], case["tokens"] * case["top"], case["n"]
        if not case["train"]:
            return {"bytes": e * n * (m + t) + 8 * m, "flops": 2 * m * n}
        # X, dout, weights, slots and rows in; out, dX and dw out
        return {"bytes": e * n * (2 * m + 2 * t) + 16 * m, "flops": 5 * m * n}
    k, n = case["k"], case["n"]
    if kind == "adapters":
        m, r = case["rows"], case["rank"]
        with_one = m * (1 - case["plain"])
        active = _reached(case["adapters"], with_one, 1 / case["adapters"])
        return {"bytes": int(e * (n * k + m * k + active * r * (k + n)) +
                             SIZE[case["out"]] * m * n + 4 * m),
                "flops": int(2 * m * n * k + 2 * with_one * r * (k + n))}
    m = case["tokens"] * case["top"]
    active = _reached(case["groups"], case["tokens"], case["top"] / case["groups"])
    if kind == "experts":
        return {"bytes": int(e * (case["tokens"] * k + active * n * k) +
                             SIZE[case["out"]] * m * n + 4 * m), "flops": 2 * m * n * k}
    # x, B, dD in; D, dA (a row per choice), dB (every expert's) out
    return {"bytes": int(e * (case["tokens"] * k + active * n * k + m * (2 * n + k) +
                              case["groups"] * n * k) + 4 * m),
            "flops": 6 * m * n * k}


# ------------------------------------------------------------------ inputs
def _choices(gen, tokens, top, groups, skew):
    """(tokens, top) different experts per token, the first ones likelier."""
    score = torch.randn(tokens, groups, generator=gen, device="cuda")
    score -= skew * torch.arange(groups, device="cuda").float().mul(8.0 / groups).sqrt()
    return score.topk(top, dim=1).indices


def _grouping(ids, groups):
    """rows, offsets and slots of `ids` (n, top): row n // top of every choice
    in the order of their groups, where each group starts, each choice's
    place (-1: no group)."""
    flat = ids.reshape(-1).long()
    n, top = flat.shape[0], ids[0].numel()
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    held, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(held, torch.arange(groups + 1, device=ids.device))
    place = torch.empty_like(order)
    place[order] = torch.arange(n, device=ids.device)
    slots = torch.where(key < groups, place, -1)
    return ((order // top).to(torch.int32), offsets.to(torch.int32),
            slots.to(torch.int32).view(ids.shape))


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    kind = case["kind"]
    s = dict(case=case)
    if kind == "order":
        ids = _choices(gen, case["tokens"], case["top"], case["groups"], case["skew"])
        away = torch.rand(case["tokens"], generator=gen, device=dev) < case["padded"]
        ids = torch.where(away[:, None], -1, ids)
        s["ids"] = ids.to(DTYPES[case["ids"]])
        return s
    dt = DTYPES[case["dtype"]]

    def values(*shape, gain=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * gain).to(dt)

    if kind == "combine":
        t, top, n = case["tokens"], case["top"], case["n"]
        m = t * top
        place = torch.randperm(m, generator=gen, device=dev)
        drop = torch.rand(m, generator=gen, device=dev) < case["missing"]
        # dropped choices lie behind the kept ones, as those of no group do
        order = place[torch.sort(drop[place].int(), stable=True).indices]
        slots = torch.empty_like(order)
        slots[order] = torch.arange(m, device=dev)
        s["rows"] = (order // top).to(torch.int32)
        s["slots"] = torch.where(drop, -1, slots).to(torch.int32).view(t, top)
        s["X"] = values(m, n)
        s["weights"] = torch.softmax(torch.randn(t, top, generator=gen, device=dev), 1)
        if case["train"]:
            s["dout"] = values(t, n)
        return s
    k, n = case["k"], case["n"]
    if kind == "adapters":
        m, r, a = case["rows"], case["rank"], case["adapters"]
        ids = torch.randint(0, a, (m,), generator=gen, device=dev)
        ids = torch.where(torch.rand(m, generator=gen, device=dev) < case["plain"], -1, ids)
        if case["runs"]:        # whole prompts: rows of a request follow each other
            ids = torch.sort(ids, stable=True).values
        s["rows"], s["offsets"], _ = _grouping(ids.view(m, 1), a)
        s["longest"] = max(1, int(s["offsets"].diff().max()))
        s["x"] = values(m, k)
        s["W"] = values(n, k, gain=k ** -0.5)
        s["A"] = values(a, r, k, gain=k ** -0.5)
        s["B"] = values(a, n, r, gain=r ** -0.5)
        s["scale"] = torch.rand(a, generator=gen, device=dev) + 0.5
        return s
    ids = _choices(gen, case["tokens"], case["top"], case["groups"], case["skew"])
    s["rows"], s["offsets"], _ = _grouping(ids, case["groups"])
    s["longest"] = int(s["offsets"].diff().max())
    s["x"] = values(case["tokens"], k)
    s["B"] = values(case["groups"], n, k, gain=k ** -0.5)
    if kind == "train":
        s["dD"] = values(ids.numel(), n)
    return s


# -------------------------------------------------------------- plain form
def _places(s):
    """Places (groups, longest) of the groups' rows, and which hold one."""
    at = s["offsets"][:-1, None].long() + torch.arange(s["longest"], device="cuda")
    held = at < s["offsets"][1:, None]
    return at.clamp(max=max(0, s["rows"].shape[0] - 1)), held


def _plain_experts(s, train):
    at, held = _places(s)
    dt = s["x"].dtype
    x = s["x"].float()[s["rows"].long()[at]] * held[..., None]
    b = s["B"].float()
    out = torch.matmul(x, b.transpose(1, 2).contiguous())[held]
    if not train:
        return out.to(DTYPES[s["case"]["out"]])
    d = s["dD"].float()[at] * held[..., None]
    dA = torch.matmul(d, b)[held]
    dB = torch.matmul(d.transpose(1, 2).contiguous(), x)
    return {"D": out.to(dt), "dA": dA.to(dt), "dB": dB.to(dt)}


def _plain_combine(s):
    X, slots, w = s["X"].float(), s["slots"].long(), s["weights"]
    dt, kept = s["X"].dtype, s["slots"] >= 0
    each = X[slots.clamp(min=0)]
    out = (each * (w * kept)[..., None]).sum(1).to(dt)
    if not s["case"]["train"]:
        return out
    dout = s["dout"].float()[:, None]
    dX = torch.zeros_like(X)
    dX[slots[kept]] = (w[..., None] * dout)[kept]
    dw = (each * dout).sum(-1) * kept
    return {"out": out, "dX": dX.to(dt), "dw": dw}


def _plain_adapters(s):
    at, held = _places(s)
    at = s["rows"].long()[at]
    x = s["x"].float()
    y = torch.matmul(x, s["W"].float().t().contiguous())
    h = torch.matmul(x[at] * held[..., None], s["A"].float().transpose(1, 2).contiguous())
    h = h * s["scale"][:, None, None]
    low = torch.matmul(h, s["B"].float().transpose(1, 2).contiguous())
    y[at[held]] += low[held]
    return y.to(DTYPES[s["case"]["out"]])


# --------------------------------------------------------------------- run
def _own_run(s):
    import mma_fragment_layouts_tn_amd as mfl

    case = s["case"]
    kind = case["kind"]
    if kind == "order":
        return list(mfl.group_rows(s["ids"], case["groups"]))
    if kind == "combine":
        out = mfl.combine_rows(s["X"], s["slots"], s["weights"])
        if not case["train"]:
            return out
        dX, dw = mfl.combine_rows_backward(s["dout"], s["X"], s["slots"], s["weights"],
                                           rows=s["rows"])
        return {"out": out, "dX": dX, "dw": dw}
    if kind == "adapters":
        return mfl.gemm_adapters(s["x"], s["W"], s["A"], s["B"], s["offsets"], rows=s["rows"],
                                 scale=s["scale"], out_dtype=DTYPES[case["out"]])
    if kind == "experts":
        return mfl.gemm_grouped(s["x"], s["B"], s["offsets"], rows=s["rows"],
                                out_dtype=DTYPES[case["out"]])
    out = mfl.gemm_grouped(s["x"], s["B"], s["offsets"], rows=s["rows"])
    dA, dB = mfl.gemm_grouped_backward(s["dD"], s["x"], s["B"], s["offsets"], rows=s["rows"])
    return {"D": out, "dA": dA, "dB": dB}


def run(s):
    if own:
        return _own_run(s)
    kind = s["case"]["kind"]
    if kind == "order":
        return list(_grouping(s["ids"], s["case"]["groups"]))
    if kind == "combine":
        return _plain_combine(s)
    if kind == "adapters":
        return _plain_adapters(s)
    return _plain_experts(s, kind == "train")


# ------------------------------------------------------------------- exact
def exact(case, seed):
    kind = case["kind"]
    if kind == "order":
        return None              # whole numbers
    s = prepare(case, seed)
    f8 = dict(dtype=torch.float64, device="cuda")
    if kind == "combine":
        X, w = s["X"].double(), s["weights"].double()
        out = torch.zeros(case["tokens"], case["n"], **f8)
        dX, dw = torch.zeros_like(X), torch.zeros_like(w)
        for j in range(case["top"]):
            slot = s["slots"][:, j].long()
            t = torch.nonzero(slot >= 0).flatten()
            row = slot[t]
            out[t] += w[t, j, None] * X[row]
            if case["train"]:
                d = s["dout"].double()[t]
                dX[row] = w[t, j, None] * d
                dw[t, j] = (d * X[row]).sum(-1)
        return {"out": out, "dX": dX, "dw": dw} if case["train"] else out
    offsets, rows, x = s["offsets"].tolist(), s["rows"].long(), s["x"].double()
    if kind == "adapters":
        y = torch.mm(x, s["W"].double().t())
        for g in range(case["adapters"]):
            at = rows[offsets[g]:offsets[g + 1]]
            low = torch.mm(x[at], s["A"][g].double().t())
            y[at] += s["scale"][g].double() * torch.mm(low, s["B"][g].double().t())
        return y
    m, train = rows.shape[0], kind == "train"
    out, dA = torch.zeros(m, case["n"], **f8), None
    if train:
        dA, dB = torch.zeros(m, case["k"], **f8), torch.zeros(s["B"].shape, **f8)
    for g in range(case["groups"]):
        a, b = offsets[g], offsets[g + 1]
        w, xg = s["B"][g].double(), x[rows[a:b]]
        out[a:b] = torch.mm(xg, w.t())
        if train:
            d = s["dD"][a:b].double()
            dA[a:b] = torch.mm(d, w)
            dB[g] = torch.mm(d.t(), xg)
    return {"D": out, "dA": dA, "dB": dB} if train else out
