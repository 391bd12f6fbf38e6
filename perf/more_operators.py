"""Cases and plain forms of the operators of a student that reads tokens: the embedding with its gradient by sorted
tokens, layer norm, and the gated delta rule (a recurrence whose state is a matrix).

listed() names the cases, draw() gives more of the same ranges, prepare() makes what a learner has in hand, run() is
one pass (the library's calls where `own` is true, elementary torch operations otherwise), work() the bytes and
operations a pass cannot do without, exact() the same outputs from the definitions in 64 bits."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
DEV = "cuda"
CHUNK = 64  # steps that the plain form of the delta rule takes at once


def listed():
    return [
        # The tokens of one step of 512 environments: the launch is what counts.
        dict(name="lookup actors", op="lookup", tokens=512, vocab=50000, dim=256, table="f32", dtype="f32", index="i32"),
        # A learner's replayed tokens over a large vocabulary, gradient of the whole table.
        dict(name="embed tokens", op="embed", tokens=65536, vocab=65536, dim=1024, table="f32", dtype="bf16",
             index="i64", hot=0.1, padding=0.0),
        # Discrete observations: few tokens, most rows share one of them, odd width, padded sequences.
        dict(name="embed observations", op="embed", tokens=20001, vocab=501, dim=333, table="f32", dtype="f32",
             index="i32", hot=0.4, padding=0.2),
        # An actor's step.
        dict(name="norm actors", op="norm", rows=512, dim=1024, dtype="f32", train=False, affine=True),
        # The learner's rows, forward and backward.
        dict(name="norm tokens", op="norm", rows=65536, dim=2048, dtype="bf16", train=True, affine=True),
        # Odd width, an odd number of rows.
        dict(name="norm odd", op="norm", rows=4095, dim=1001, dtype="f16", train=True, affine=True),
        # One token for each of a few environments.
        dict(name="delta step few", op="step", batch=8, heads=4, qk_heads=4, dk=64, dv=64, dtype="f32"),
        # One token for each of many: every state is read and written.
        dict(name="delta step many", op="step", batch=256, heads=16, qk_heads=16, dk=128, dv=128, dtype="bf16"),
        # Replayed windows with episode borders inside them, ragged, in full precision, forward and backward.
        dict(name="delta windows", op="delta", batch=37, steps=81, heads=4, qk_heads=4, dk=48, dv=65, dtype="f32",
             train=True, ragged=True),
        # The learner's sequences, value heads that share queries and keys.
        dict(name="delta replay", op="delta", batch=32, steps=512, heads=16, qk_heads=8, dk=128, dv=128, dtype="bf16",
             train=True, ragged=False),
        # Few long sequences.
        dict(name="delta long", op="delta", batch=1, steps=16384, heads=8, qk_heads=8, dk=128, dv=128, dtype="bf16",
             train=True, ragged=False),
        # A prompt read by the serving side: the outputs and the last state alone.
        dict(name="delta prompt", op="delta", batch=4, steps=2048, heads=16, qk_heads=16, dk=128, dv=128, dtype="f16",
             train=False, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "embed", "norm", "step", "delta", "delta"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("lookup", "embed"):
        dim = _log(rng, 8, 4096)
        vocab = _log(rng, 16, min(200000, (1 << 26) // dim))
        c = dict(op=op, tokens=_log(rng, 1, min(131072, (1 << 26) // dim)), vocab=vocab, dim=dim,
                 table=rng.choice(["f32", dtype]), dtype=dtype, index=rng.choice(["i32", "i64"]))
        if op == "embed":
            c.update(hot=rng.choice([0.0, 0.1, 0.5]), padding=rng.choice([0.0, 0.3]))
        return c
    if op == "norm":
        dim = _log(rng, 8, 16384)
        return dict(op=op, rows=_log(rng, 1, min(131072, (1 << 26) // dim)), dim=dim, dtype=dtype,
                    train=rng.random() < 0.7, affine=rng.random() < 0.8)
    shared = rng.choice([1, 1, 2, 4])
    qk_heads = _log(rng, 1, 16 // shared)
    dk, dv = (rng.choice([32, 64, 128, rng.randint(8, 128)]) for _ in range(2))
    c = dict(op=op, heads=qk_heads * shared, qk_heads=qk_heads, dk=dk, dv=dv, dtype=dtype)
    if op == "step":
        c["batch"] = _log(rng, 1, max(1, (1 << 25) // (c["heads"] * dk * dv)))
        return c
    steps = _log(rng, 1, 8192)
    c.update(steps=steps, batch=_log(rng, 1, max(1, min(64, (1 << 24) // (steps * c["heads"] * (dk + dv))))),
             train=rng.random() < 0.7, ragged=rng.random() < 0.5)
    return c


# ------------------------------------------------------------------------------------------------------ inputs

def _tokens(c, g):
    """Tokens whose frequency falls with their rank, a share of them one and the same token, and padding (-1)."""
    n, v = c["tokens"], c["vocab"]
    rank = torch.exp(torch.rand(n, device=DEV, generator=g, dtype=torch.float64) * math.log(v + 1)) - 1
    mixed = torch.randperm(v, device=DEV, generator=g)
    t = mixed[rank.long().clamp(0, v - 1)]
    t = torch.where(torch.rand(n, device=DEV, generator=g) < c.get("hot", 0.0), mixed[v // 2], t)
    t = torch.where(torch.rand(n, device=DEV, generator=g) < c.get("padding", 0.0), -1, t)
    return t.to(torch.int32 if c["index"] == "i32" else torch.int64)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"c": c}
    dt = DTYPES[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    if c["op"] in ("lookup", "embed"):
        s["tokens"] = _tokens(c, g)
        s["table"] = (0.05 * randn(c["vocab"], c["dim"])).to(DTYPES[c["table"]])
        s["scale"] = math.sqrt(c["dim"])
        if c["op"] == "embed":
            s["dout"] = (1e-2 * randn(c["tokens"], c["dim"])).to(dt)
    elif c["op"] == "norm":
        n, d = c["rows"], c["dim"]
        s["x"] = (randn(n, d) * torch.exp(0.3 * randn(d)) + 0.5 * randn(n, 1)).to(dt)
        s["weight"] = 1 + 0.1 * randn(d) if c["affine"] else None
        s["bias"] = 0.1 * randn(d) if c["affine"] else None
        if c["train"]:
            s["dy"] = randn(n, d).to(dt)
    else:
        b, t, h, hk, dk, dv = c["batch"], c.get("steps", 1), c["heads"], c["qk_heads"], c["dk"], c["dv"]
        q, k = randn(b, t, hk, dk), randn(b, t, hk, dk) + 0.3 * randn(b, 1, hk, dk)
        s["q"], s["k"] = ((x / x.square().sum(-1, keepdim=True).sqrt()).to(dt) for x in (q, k))
        both = randn(b, t, h, dv + 2)  # one projection gives the values, the gates and the writing strengths
        both[..., dv] = both[..., dv] * 1.5 + 4
        both = both.to(dt)
        s["v"], s["g"], s["b"] = both[..., :dv], both[..., dv], both[..., dv + 1]
        s["scale"] = dk ** -0.5
        s["s0"] = randn(b, h, dk, dv) * dk ** -0.5
        if c["op"] == "step":
            s["q"], s["k"], s["v"], s["g"], s["b"] = (s[x][:, 0] for x in "qkvgb")
            s["reset"] = torch.rand(b, device=DEV, generator=g) < 0.02
            s["s_out"], s["o"] = torch.empty_like(s["s0"]), torch.empty(b, h, dv, dtype=dt, device=DEV)
        else:
            s["reset"] = torch.rand(b, t, device=DEV, generator=g) < 0.005
            s["length"] = torch.randint(t // 2, t + 1, (b,), device=DEV, generator=g) if c["ragged"] else None
            if c["train"]:
                s["do"] = randn(b, t, h, dv).to(dt)
                s["ds"] = randn(b, h, dk, dv) * dk ** -0.5
    return s


# ----------------------------------------------------------------------------------------------------- one pass

def run(s):
    c = s["c"]
    return {"lookup": _lookup, "embed": _embed, "norm": _norm, "step": _step, "delta": _delta}[c["op"]](s, c)


def _rows(s, c):
    tokens = s["tokens"].long()
    there = (tokens >= 0) & (tokens < c["vocab"])
    out = s["table"][tokens.clamp(0, c["vocab"] - 1)].float() * s["scale"]
    return tokens, there, torch.where(there[:, None], out, torch.zeros_like(out)).to(DTYPES[c["dtype"]])


def _lookup(s, c):
    if own:
        import sum_tree_sampling_amd as per
        return per.per_embed_forward(s["tokens"], s["table"], scale=s["scale"], dtype=DTYPES[c["dtype"]])
    return _rows(s, c)[2]


def _embed(s, c):
    if own:
        import sum_tree_sampling_amd as per
        out = per.per_embed_forward(s["tokens"], s["table"], scale=s["scale"], dtype=DTYPES[c["dtype"]])
        return {"out": out, "grad": per.per_embed_backward(s["tokens"], s["dout"], c["vocab"], scale=s["scale"])}
    tokens, there, out = _rows(s, c)
    grad = torch.zeros(c["vocab"] + 1, c["dim"], device=DEV)
    grad.index_add_(0, torch.where(there, tokens, c["vocab"]), s["dout"].float())
    return {"out": out, "grad": grad[:-1] * s["scale"]}


def _norm(s, c):
    x, weight, bias = s["x"], s["weight"], s["bias"]
    if own:
        import sum_tree_sampling_amd as per
        y, stats = per.per_norm_forward(x, weight, bias, eps=1e-5)
        if not c["train"]:
            return {"y": y}
        dx, dweight, dbias = per.per_norm_backward(x, stats, s["dy"], weight)
        return {"y": y, "dx": dx, "dweight": dweight, "dbias": dbias}
    dt = x.dtype
    x = x.float()
    d = x - x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5)
    xhat = d * rstd
    y = (xhat if weight is None else xhat * weight + bias).to(dt)
    if not c["train"]:
        return {"y": y}
    dy = s["dy"].float()
    dxhat = dy if weight is None else dy * weight
    dx = rstd * (dxhat - dxhat.mean(1, keepdim=True) - xhat * (dxhat * xhat).mean(1, keepdim=True))
    return {"y": y, "dx": dx.to(dt), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


def _sigmoid(x):
    e = torch.exp(-x.abs())
    return torch.where(x >= 0, 1 / (1 + e), e / (1 + e))


def _step(s, c):
    if own:
        import sum_tree_sampling_amd as per
        per.per_delta_step(s["q"], s["k"], s["v"], s["g"], s["b"], s["s0"], reset=s["reset"], scale=s["scale"],
                           s_out=s["s_out"], out=s["o"])
        return {"o": s["o"], "s": s["s_out"]}
    shared = c["heads"] // c["qk_heads"]
    q, k = (s[x].float().repeat_interleave(shared, 1) for x in "qk")
    f, w = _sigmoid(s["g"].float()), _sigmoid(s["b"].float())
    state = torch.where(s["reset"][:, None, None, None], torch.zeros_like(s["s0"]), s["s0"]) * f[..., None, None]
    u = w[..., None] * (s["v"].float() - (k[..., None] * state).sum(2))
    state = state + k[..., None] * u[:, :, None]
    o = (q[..., None] * state).sum(2) * s["scale"]
    return {"o": o.to(s["v"].dtype), "s": state}


def _delta(s, c):
    if own:
        import sum_tree_sampling_amd as per
        o, last, carries = per.per_delta_forward(s["q"], s["k"], s["v"], s["g"], s["b"], reset=s["reset"],
                                                 length=s["length"], s0=s["s0"], scale=s["scale"], save=c["train"])
        if not c["train"]:
            return {"o": o, "s": last}
        dq, dk, dv, dg, db, ds0 = per.per_delta_backward(s["q"], s["k"], s["v"], s["g"], s["b"], carries, s["do"],
                                                         reset=s["reset"], length=s["length"], ds_last=s["ds"],
                                                         scale=s["scale"])
        return {"o": o, "s": last, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "db": db, "ds0": ds0}
    if not c["train"]:
        o, last = _delta_plain(s, c, *(s[x] for x in ("q", "k", "v", "g", "b", "s0")))
        return {"o": o.to(s["v"].dtype), "s": last}
    ins = [s[x].float().requires_grad_() for x in ("q", "k", "v", "g", "b")]
    ins.append(s["s0"].detach().clone().requires_grad_())
    o, last = _delta_plain(s, c, *ins)
    dq, dk, dv, dg, db, ds0 = torch.autograd.grad((o, last), ins, (s["do"].float(), s["ds"]))
    dt = s["v"].dtype
    return {"o": o.detach().to(dt), "s": last.detach(), "dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt),
            "dg": dg.to(dt), "db": db.to(dt), "ds0": ds0}


def _delta_plain(s, c, q, k, v, g, b, state):
    """The delta rule in chunks: inside one, the rows that the state takes up are u = (I + A)^-1 (w v - w decay k S),
    with A the products of its keys below the diagonal; from chunk to chunk the state is carried on."""
    B, T, H = v.shape[:3]
    n = -(-T // CHUNK)
    shared = H // q.shape[2]
    live = torch.arange(n * CHUNK, device=DEV) < (s["length"][:, None] if s["length"] is not None else T)

    def chunks(x):  # [B x T x H x ...] to [B x H x n x CHUNK x ...], zeros where nothing is
        x = torch.cat([x, x.new_zeros(B, n * CHUNK - T, *x.shape[2:])], 1)
        x = torch.where(live.view(B if live.dim() == 2 else 1, -1, *[1] * (x.dim() - 2)), x, torch.zeros_like(x))
        return x.movedim(1, 2).reshape(B, x.shape[2], n, CHUNK, *x.shape[3:])

    q, k = (chunks(x.float()).repeat_interleave(shared, 1) for x in (q, k))
    v = chunks(v.float())
    g = g.double()
    decay = chunks(-torch.clamp(-g, min=0) - torch.log(1 + torch.exp(-g.abs()))).cumsum(3)  # log, from the chunk's begin
    w = chunks(_sigmoid(b.float()))
    seen = chunks(s["reset"][..., None].long()).cumsum(3)  # resets up to a step
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    gap = torch.where((seen[..., None] == seen[..., None, :]) & lower, decay[..., None] - decay[..., None, :], -math.inf)
    between = torch.exp(gap).float()
    first = torch.exp(torch.where(seen == 0, decay, -math.inf)).float()[..., None]
    last = torch.exp(torch.where(seen == seen[..., -1:], decay[..., -1:] - decay, -math.inf)).float()[..., None]
    a = w[..., None] * (k @ k.transpose(-1, -2)) * between
    # (I + A)^-1 from blocks of one row, two blocks joined at a time
    at = torch.arange(CHUNK, device=DEV)
    inv = torch.eye(CHUNK, device=DEV).expand_as(a)
    size = 1
    while size < CHUNK:
        join = (at[:, None] // size == at // size + 1) & (at // size % 2 == 0)
        inv = inv - inv @ torch.where(join, a, torch.zeros_like(a)) @ inv
        size *= 2
    scores = (q @ k.transpose(-1, -2)) * between
    write, read = (k * last).transpose(-1, -2), k * first
    asked = q * first
    outs = []
    rows = zip(*(x.unbind(2) for x in (inv, w[..., None], v, read, asked, scores, write, first[:, :, :, -1:])))
    for inv, w, v, read, asked, scores, write, kept in rows:  # the states follow each other
        u = inv @ (w * (v - read @ state))
        outs.append(asked @ state + scores @ u)
        state = kept * state + write @ u
    o = torch.stack(outs, 2) * s["scale"]
    return o.reshape(B, H, n * CHUNK, -1)[:, :, :T].movedim(2, 1), state


# --------------------------------------------------------------------------------------------------- the work

def work(case):
    c, size = case, SIZE[case["dtype"]]
    if c["op"] in ("lookup", "embed"):
        n = c["tokens"] * c["dim"]
        index = c["tokens"] * (4 if c["index"] == "i32" else 8)
        most = min(c["tokens"], c["vocab"]) * c["dim"]  # rows of the table, each read once
        look = most * SIZE[c["table"]] + n * size + index
        if c["op"] == "lookup":
            return {"bytes": look, "flops": n}
        return {"bytes": look + n * size + 4 * c["vocab"] * c["dim"] + index, "flops": 3 * n}
    if c["op"] == "norm":
        n = c["rows"] * c["dim"]
        if not c["train"]:
            return {"bytes": 2 * n * size + 8 * c["dim"], "flops": 8 * n}
        return {"bytes": 5 * n * size + 28 * c["dim"] + 16 * c["rows"], "flops": 22 * n}
    states = c["batch"] * c["heads"] * c["dk"] * c["dv"]
    rows = c["batch"] * c.get("steps", 1)
    io = rows * (2 * c["qk_heads"] * c["dk"] + c["heads"] * (c["dv"] + 2)) * size  # q, k, v, g, b
    o = rows * c["heads"] * c["dv"] * size
    n = rows * c["heads"] * c["dk"] * c["dv"]
    if c["op"] == "step" or not c["train"]:
        return {"bytes": io + o + 8 * states, "flops": 7 * n}  # decay, k S, k u, q S
    return {"bytes": 3 * io + 2 * o + 16 * states, "flops": 22 * n}


# ------------------------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"lookup": _exact_embed, "embed": _exact_embed, "norm": _exact_norm, "step": _exact_step,
            "delta": _exact_delta}[case["op"]](s, case)


def _exact_embed(s, c):
    tokens = s["tokens"].long()
    there = (tokens >= 0) & (tokens < c["vocab"])
    out = torch.zeros(c["tokens"], c["dim"], dtype=torch.float64, device=DEV)
    out[there] = s["table"][tokens[there]].double() * s["scale"]
    if c["op"] == "lookup":
        return out
    order = torch.argsort(tokens[there], stable=True)
    rows = s["dout"][there][order]
    token, count = torch.unique_consecutive(tokens[there][order], return_counts=True)
    grad = torch.zeros(c["vocab"], c["dim"], dtype=torch.float64, device=DEV)
    ends = count.cumsum(0)
    width = max(1, (1 << 26) // max(1, rows.shape[0]))
    for lo in range(0, c["dim"], width):  # sums of a token's rows by differences of running sums
        total = torch.cat([rows.new_zeros(1, min(width, c["dim"] - lo), dtype=torch.float64),
                           rows[:, lo:lo + width].double().cumsum(0)])
        grad[token, lo:lo + width] = (total[ends] - total[ends - count]) * s["scale"]
    return {"out": out, "grad": grad}


def _exact_norm(s, c):
    x = s["x"].double()
    weight = s["weight"].double() if c["affine"] else torch.ones(c["dim"], dtype=torch.float64, device=DEV)
    var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
    sigma = (var + 1e-5).sqrt()
    h = (x - mean) / sigma
    y = h * weight + (s["bias"].double() if c["affine"] else 0)
    if not c["train"]:
        return {"y": y}
    dy = s["dy"].double()
    e = dy * weight
    n = c["dim"]
    dx = (n * e - e.sum(1, keepdim=True) - h * (e * h).sum(1, keepdim=True)) / (n * sigma)
    return {"y": y, "dx": dx, "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}


def _exact_step(s, c):
    shared = c["heads"] // c["qk_heads"]
    q, k = (s[x].double().repeat_interleave(shared, 1) for x in "qk")
    f, w = (1 / (1 + torch.exp(-s[x].double())) for x in "gb")
    state = s["s0"].double() * f[..., None, None]
    state[s["reset"]] = 0
    u = w[..., None] * (s["v"].double() - torch.einsum("bhkv,bhk->bhv", state, k))
    state = state + torch.einsum("bhk,bhv->bhkv", k, u)
    return {"o": s["scale"] * torch.einsum("bhkv,bhk->bhv", state, q), "s": state}


def _exact_delta(s, c):
    B, T, H, hk, scale = c["batch"], c["steps"], c["heads"], c["qk_heads"], s["scale"]
    if B * H * c["dk"] * c["dv"] * 8 * 66 > 40e9:
        return None
    q, k, v, f, w = (s[x].double() for x in "qkvgb")
    q, k = (x.repeat_interleave(H // hk, 2) for x in (q, k))
    f, w = 1 / (1 + torch.exp(-f)), 1 / (1 + torch.exp(-w))
    n = s["length"] if c["ragged"] else torch.full((B,), T, device=DEV)
    go = (torch.arange(T, device=DEV) < n[:, None]).double()
    # a step that is not there keeps the state: gate 1, nothing written; a reset: gate 0
    keep = torch.where(s["reset"], 0.0, 1.0).double()
    gate = torch.where(go[..., None] > 0, f * keep[..., None], torch.ones_like(f))
    w_, f_ = w * go[..., None], f
    k = k * go[..., None, None]

    def advance(state, t):
        before = state * gate[:, t, :, None, None]
        r = v[:, t] - (before * k[:, t, :, :, None]).sum(2)
        u = w_[:, t, :, None] * r
        return before, r, u, before + k[:, t, :, :, None] * u[:, :, None]

    state, o, held = s["s0"].double(), torch.zeros(v.shape, dtype=torch.float64, device=DEV), []
    for t in range(T):
        if t % 64 == 0:
            held.append(state)
        state = advance(state, t)[3]
        o[:, t] = scale * go[:, t, None, None] * (state * q[:, t, :, :, None]).sum(2)
    if not c["train"]:
        return {"o": o, "s": state}
    do = s["do"].double() * go[..., None, None]
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    dg, db = torch.zeros_like(f), torch.zeros_like(w)
    ds = s["ds"].double()
    for first in reversed(range(0, T, 64)):
        x, steps = held.pop(), []
        for t in range(first, min(T, first + 64)):
            steps.append((x,) + advance(x, t))
            x = steps[-1][4]
        for t in reversed(range(first, min(T, first + 64))):
            past, before, r, u, after = steps.pop()
            dq[:, t] = scale * (after * do[:, t, :, None]).sum(3)
            ds = ds + scale * q[:, t, :, :, None] * do[:, t, :, None]
            du = (ds * k[:, t, :, :, None]).sum(2)
            dr = w_[:, t, :, None] * du
            dk[:, t] = (ds * u[:, :, None]).sum(3) - (before * dr[:, :, None]).sum(3)
            dv[:, t] = dr
            db[:, t] = (du * r).sum(2) * w[:, t] * (1 - w[:, t])
            ds = ds - k[:, t, :, :, None] * dr[:, :, None]
            dg[:, t] = (ds * past).sum((2, 3)) * (keep[:, t] * go[:, t])[:, None] * f_[:, t] * (1 - f_[:, t])
            ds = ds * gate[:, t, :, None, None]
    on = go[..., None]
    dq, dk = ((x * on[..., None]).view(B, T, hk, H // hk, -1).sum(3) for x in (dq, dk))
    return {"o": o, "s": state, "dq": dq, "dk": dk, "dv": dv, "dg": dg * on, "db": db * on, "ds0": ds}
