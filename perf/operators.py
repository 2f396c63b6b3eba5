"""Cases of the attention operators: whole prompts, a training step, and
decoding behind a shared prefix.

Each case names its kind:

  prompt   attention() over packed prompts (or chunks of them), one pass
  train    attention() with its log-sum-exp, then attention_backward()
  prefix   attention_prefix(): one step of a decoding batch whose sequences
           share a prefix

`run` takes the plain form below, or with `own` the framework's entry points.
The plain form pads the packed batch, masks, and uses matrix products, exp
and sums in float32; `exact` is the definition in float64, sequence by
sequence.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the first tokens of a short chat turn: latency counts
        dict(name="prompt_short", kind="prompt", dtype="bf16", heads=32, kv_heads=8, dim=128,
             q_lens="128", k_lens="128", causal=True),
        # a serving batch of prompts of very different lengths, one of a single token
        dict(name="prompt_packed", kind="prompt", dtype="bf16", heads=32, kv_heads=8, dim=128,
             q_lens="2048,1,731,4096,17,1500,300,33", k_lens="2048,1,731,4096,17,1500,300,33",
             causal=True),
        # one long document
        dict(name="prompt_long", kind="prompt", dtype="f16", heads=32, kv_heads=8, dim=128,
             q_lens="8192", k_lens="8192", causal=True),
        # chunks of prompts whose earlier tokens are in the cache already
        dict(name="prompt_chunked", kind="prompt", dtype="bf16", heads=16, kv_heads=16, dim=64,
             q_lens="512,100,1,256", k_lens="8192,4001,2500,256", causal=True),
        # a bidirectional encoder's batch, no mask
        dict(name="prompt_encoder", kind="prompt", dtype="f16", heads=16, kv_heads=16, dim=64,
             q_lens="512,384,512,77,512,129,500,512", k_lens="512,384,512,77,512,129,500,512",
             causal=False),
        # fine-tuning on a few short samples
        dict(name="train_short", kind="train", dtype="bf16", heads=16, kv_heads=4, dim=128,
             q_lens="200,333,512", k_lens="200,333,512", causal=True),
        # pretraining on packed documents
        dict(name="train_packed", kind="train", dtype="bf16", heads=32, kv_heads=8, dim=128,
             q_lens="4096,1021,2048,1027", k_lens="4096,1021,2048,1027", causal=True),
        # an encoder's or cross-attention's training step, small heads
        dict(name="train_encoder", kind="train", dtype="f16", heads=16, kv_heads=16, dim=64,
             q_lens="1024,1024,2000", k_lens="1024,1500,2000", causal=False),
        # two answers sampled behind one system prompt
        dict(name="prefix_two", kind="prefix", dtype="bf16", heads=32, kv_heads=8, dim=128,
             batch=2, q_tokens=1, prefix=1000, capacity=512, least=1, most=200),
        # a serving batch behind a shared instruction
        dict(name="prefix_batch", kind="prefix", dtype="bf16", heads=32, kv_heads=8, dim=128,
             batch=64, q_tokens=1, prefix=8192, capacity=1024, least=0, most=1000),
        # many samples of one long context
        dict(name="prefix_long", kind="prefix", dtype="f16", heads=32, kv_heads=8, dim=128,
             batch=128, q_tokens=1, prefix=32768, capacity=2048, least=256, most=2048),
        # drafted tokens checked together, every head with its own cache
        dict(name="prefix_draft", kind="prefix", dtype="bf16", heads=16, kv_heads=16, dim=64,
             batch=16, q_tokens=4, prefix=2047, capacity=640, least=4, most=600),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "train", "prefix", "prefix"])
    case = dict(kind=kind, dtype=rng.choice(["bf16", "f16"]),
                dim=rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 256]))
    case["kv_heads"] = rng.choice([1, 2, 4, 8, 16])
    case["heads"] = min(32, case["kv_heads"] * rng.choice([1, 2, 4, 8]))
    if kind == "prefix":
        case["batch"] = _log_int(rng, 1, 128)
        case["q_tokens"] = rng.choice([1, 1, 1, 2, 5])
        case["prefix"] = _log_int(rng, 64, 16384)
        case["capacity"] = _log_int(rng, 16, 1024)
        case["most"] = case["capacity"]
        case["least"] = rng.randint(0, min(case["q_tokens"], case["most"]))
        return case
    case["causal"] = rng.random() < 0.75
    count = _log_int(rng, 1, 16)
    longest = _log_int(rng, 64, 8192 if count == 1 else 4096 if count <= 3 else 1536)
    if kind == "train" or case["dim"] == 256:
        longest = min(longest, 2560)
    k = [longest] + [_log_int(rng, 1, longest) for _ in range(count - 1)]
    rng.shuffle(k)
    q = list(k)
    other = rng.random()
    if other < 0.4:             # chunks of prompts
        q = [rng.randint(1, n) for n in k]
    elif other < 0.5:           # queries of another text: causal rows may see nothing
        q = [rng.randint(1, longest) for _ in k]
    case["q_lens"] = ",".join(map(str, q))
    case["k_lens"] = ",".join(map(str, k))
    return case


def _lens(text):
    return [int(x) for x in text.split(",")]


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    n = 0
    for lq, lk in zip(_lens(case["q_lens"]), _lens(case["k_lens"])):
        if not case["causal"]:
            n += lq * lk
        else:                    # query t sees keys 0 .. t + lk - lq
            first = max(0, lq - lk)
            n += sum(range(first + lk - lq + 1, lk + 1)) if lk else 0
    return n


def _own_lengths(case, gen):
    return torch.randint(case["least"], case["most"] + 1, (case["batch"],), generator=gen)


def work(case):
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["kind"] == "prefix":
        rows = case["batch"] * case["q_tokens"] * h
        mean = (case["least"] + case["most"]) / 2
        keys = case["prefix"] + case["batch"] * mean
        return {"bytes": int(2 * d * (2 * rows + 2 * hk * keys) + 4 * rows),
                "flops": int(4 * d * rows * (case["prefix"] + mean))}
    tq, tk = sum(_lens(case["q_lens"])), sum(_lens(case["k_lens"]))
    q, kv, lse = 2 * d * h * tq, 2 * d * hk * tk, 4 * h * tq
    if case["kind"] == "prompt":
        return {"bytes": 2 * q + 2 * kv, "flops": 4 * d * h * _pairs(case)}
    # q, k, v, dout in; out, lse, dq, dk, dv out
    return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * d * h * _pairs(case)}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)

    def values(*shape, gain=1.0):
        x = torch.randn(*shape, generator=gen, device=dev)
        return (x * gain).to(dt)

    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    s = dict(case=case, scale=d ** -0.5)
    if case["kind"] == "prefix":
        b, tq, cap = case["batch"], case["q_tokens"], case["capacity"]
        s["q"] = values(b, tq, h, d, gain=2.0)
        s["prefix_k"], s["prefix_v"] = values(case["prefix"], hk, d), values(case["prefix"], hk, d)
        s["k"], s["v"] = values(b, cap, hk, d), values(b, cap, hk, d)
        s["lengths"] = _own_lengths(case, host).to(torch.int32).to(dev)
        return s
    ql, kl = _lens(case["q_lens"]), _lens(case["k_lens"])
    s["q"] = values(sum(ql), h, d, gain=2.0)
    s["k"], s["v"] = values(sum(kl), hk, d), values(sum(kl), hk, d)
    s["seq_q"] = torch.tensor([0] + ql).cumsum(0).to(torch.int32).to(dev)
    s["seq_k"] = torch.tensor([0] + kl).cumsum(0).to(torch.int32).to(dev)
    s["max_q"], s["max_k"] = max(ql), max(kl)
    if case["kind"] == "train":
        s["dout"] = values(sum(ql), h, d)
    return s


# -------------------------------------------------------------- plain form
def _pad(x, seq, longest):
    """(tokens, heads, dim) -> (batch, heads, longest, dim) float32, zeros
    behind each sequence; and which places hold a token."""
    at = seq[:-1, None].long() + torch.arange(longest, device=x.device)
    held = at < seq[1:, None]
    y = x.float()[at.clamp(max=x.shape[0] - 1)] * held[..., None, None]
    return y.transpose(1, 2).contiguous(), held


def _padded(s):
    """q as (batch, kv heads, group, len, dim), k and v as (batch, kv heads,
    1, len, dim), and the mask of visible pairs (batch, len, len)."""
    case = s["case"]
    hk, g = case["kv_heads"], case["heads"] // case["kv_heads"]
    q, in_q = _pad(s["q"], s["seq_q"], s["max_q"])
    k, in_k = _pad(s["k"], s["seq_k"], s["max_k"])
    v, _ = _pad(s["v"], s["seq_k"], s["max_k"])
    q = q.unflatten(1, (hk, g)).flatten(2, 3)       # group x len rows of one kv head
    seen = in_q[:, :, None] & in_k[:, None, :]
    if case["causal"]:
        lq, lk = s["seq_q"].diff(), s["seq_k"].diff()
        i = torch.arange(s["max_q"], device=q.device)[:, None]
        j = torch.arange(s["max_k"], device=q.device)[None, :]
        seen = seen & (j <= i + (lk - lq)[:, None, None])
    return q, k, v, seen, in_q


def _softmax(scores, seen):
    """Weights and log-sum-exp over the last axis; rows that see nothing get
    weights 0 and -inf."""
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = top + total.log()
    p /= torch.where(total == 0, torch.ones_like(total), total)
    return p, lse.squeeze(-1)


def _unpad(x, held, heads):
    """(batch, kv heads, group x len, dim) -> (tokens, heads, dim)."""
    b, _, _, d = x.shape
    return x.reshape(b, heads, -1, d).transpose(1, 2)[held]


def _plain_packed(s, train):
    case, scale = s["case"], s["scale"]
    h, hk = case["heads"], case["kv_heads"]
    g = h // hk
    q, k, v, seen, in_q = _padded(s)
    b, lq, lk = q.shape[0], s["max_q"], s["max_k"]
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(scale)
    p, lse = _softmax(scores.view(b, hk, g, lq, lk), seen[:, None, None])
    p = p.view(b, hk, g * lq, lk)
    out = torch.matmul(p, v)
    dt = s["q"].dtype
    if not train:
        return _unpad(out, in_q, h).to(dt)
    lse = lse.reshape(b, h, lq).transpose(1, 2)[in_q]
    dout, _ = _pad(s["dout"], s["seq_q"], lq)
    dout = dout.unflatten(1, (hk, g)).flatten(2, 3)
    in_k = torch.arange(lk, device=q.device) < s["seq_k"].diff()[:, None]
    dv = torch.matmul(p.transpose(-1, -2).contiguous(), dout)
    ds = torch.matmul(dout, v.transpose(-1, -2).contiguous())
    ds = ds.sub_((dout * out).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    del p
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2).contiguous(), q)
    return {"out": _unpad(out, in_q, h).to(dt), "lse": lse, "dq": _unpad(dq, in_q, h).to(dt),
            "dk": _unpad(dk, in_k, hk).to(dt), "dv": _unpad(dv, in_k, hk).to(dt)}


def _plain_prefix(s):
    case = s["case"]
    b, tq, h, hk, d = (case[x] for x in ("batch", "q_tokens", "heads", "kv_heads", "dim"))
    g = h // hk
    q = s["q"].float().unflatten(2, (hk, g)).permute(2, 0, 3, 1, 4)       # hk, b, g, tq, d
    q = q.contiguous() * s["scale"]
    pk = s["prefix_k"].float().permute(1, 2, 0).contiguous()              # hk, d, P
    pv = s["prefix_v"].float().transpose(0, 1).contiguous()               # hk, P, d
    k = s["k"].float().permute(2, 0, 3, 1).contiguous()                   # hk, b, d, S
    v = s["v"].float().permute(2, 0, 1, 3).contiguous()                   # hk, b, S, d
    shared = torch.matmul(q.view(hk, b * g * tq, d), pk).view(hk, b, g, tq, -1)
    mine = torch.matmul(q.view(hk, b, g * tq, d), k).view(hk, b, g, tq, -1)
    j = torch.arange(case["capacity"], device=q.device)
    t = torch.arange(tq, device=q.device)
    seen = j <= (s["lengths"][:, None, None] - tq + t[:, None])           # b, tq, S
    seen = torch.cat([seen.new_ones(b, tq, case["prefix"]), seen], -1)[:, None]
    p, lse = _softmax(torch.cat([shared, mine], -1), seen)
    a, c = p[..., :case["prefix"]], p[..., case["prefix"]:]
    out = torch.matmul(a.reshape(hk, b * g * tq, -1), pv).view(hk, b, g, tq, d)
    out = out + torch.matmul(c.reshape(hk, b, g * tq, -1), v).view(hk, b, g, tq, d)
    out = out.permute(1, 3, 0, 2, 4).reshape(b, tq, h, d)
    lse = lse.permute(1, 3, 0, 2).reshape(b, tq, h)
    return {"out": out.to(s["q"].dtype), "lse": lse}


# --------------------------------------------------------------------- run
def _own_run(s):
    import mma_fragment_layouts_tn_amd as mfl

    case = s["case"]
    if case["kind"] == "prefix":
        out, lse = mfl.attention_prefix(s["q"], s["prefix_k"], s["prefix_v"], s["k"], s["v"],
                                        s["lengths"], scale=s["scale"], return_lse=True)
        return {"out": out, "lse": lse}
    how = dict(seq_q=s["seq_q"], seq_k=s["seq_k"], causal=case["causal"], scale=s["scale"])
    if case["kind"] == "prompt":
        return mfl.attention(s["q"], s["k"], s["v"], **how)
    out, lse = mfl.attention(s["q"], s["k"], s["v"], return_lse=True, **how)
    dq, dk, dv = mfl.attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, **how)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def run(s):
    if own:
        return _own_run(s)
    if s["case"]["kind"] == "prefix":
        return _plain_prefix(s)
    return _plain_packed(s, s["case"]["kind"] == "train")


# ------------------------------------------------------------------- exact
def _attend(q, k, v, limit, scale):
    """One head, float64: q (n, d), k and v (m, d); row i sees keys
    0 .. limit[i].  Returns out, lse and the weights."""
    z = torch.mm(q, k.t()) * scale
    hidden = torch.arange(k.shape[0], device=q.device)[None, :] > limit[:, None]
    lse = torch.logsumexp(z.masked_fill_(hidden, -math.inf), -1)
    w = torch.exp(z - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return torch.mm(w, v), lse, w


def _exact_prefix(s):
    case = s["case"]
    b, tq, h, hk = (case[x] for x in ("batch", "q_tokens", "heads", "kv_heads"))
    g = h // hk
    n = s["lengths"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(b, tq, h, dtype=torch.float64, device="cuda")
    back = torch.arange(tq, device="cuda") - tq + 1
    for kv in range(hk):
        heads = slice(kv * g, kv * g + g)
        pk, pv = s["prefix_k"][:, kv].double(), s["prefix_v"][:, kv].double()
        for i in range(b):
            k = torch.cat([pk, s["k"][i, :n[i], kv].double()])
            v = torch.cat([pv, s["v"][i, :n[i], kv].double()])
            rows = s["q"][i, :, heads].double().flatten(0, 1)
            own_last = (back + n[i] - 1).clamp(min=-1) + case["prefix"]
            o, z, _ = _attend(rows, k, v, own_last.repeat_interleave(g), s["scale"])
            out[i, :, heads] = o.view(tq, g, -1)
            lse[i, :, heads] = z.view(tq, g)
    return {"out": out, "lse": lse}


def _exact_packed(s, train):
    case, scale = s["case"], s["scale"]
    h, hk = case["heads"], case["kv_heads"]
    g = h // hk
    f8 = dict(dtype=torch.float64, device="cuda")
    out = torch.zeros(s["q"].shape, **f8)
    lse = torch.zeros(out.shape[:2], **f8)
    dq, dk, dv = torch.zeros_like(out), torch.zeros(s["k"].shape, **f8), torch.zeros(s["v"].shape, **f8)
    q0 = k0 = 0
    for lq, lk in zip(_lens(case["q_lens"]), _lens(case["k_lens"])):
        a, c = slice(q0, q0 + lq), slice(k0, k0 + lk)
        q0, k0 = q0 + lq, k0 + lk
        last = torch.arange(lq, device="cuda") + lk - lq if case["causal"] else \
            torch.full((lq,), lk, device="cuda")
        for x in range(h):
            q, k, v = (y.double() for y in (s["q"][a, x], s["k"][c, x // g], s["v"][c, x // g]))
            o, z, w = _attend(q, k, v, last, scale)
            out[a, x], lse[a, x] = o, z
            if not train:
                continue
            do = s["dout"][a, x].double()
            dv[c, x // g] += torch.mm(w.t(), do)
            dw = torch.mm(do, v.t())
            dz = w * (dw - (w * dw).sum(-1, keepdim=True)) * scale
            dq[a, x] = torch.mm(dz, k)
            dk[c, x // g] += torch.mm(dz.t(), q)
    if not train:
        return out
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "prefix":
        if case["batch"] * case["kv_heads"] * (case["prefix"] + case["most"]) > 5e7:
            return None
        return _exact_prefix(s)
    return _exact_packed(s, case["kind"] == "train")
