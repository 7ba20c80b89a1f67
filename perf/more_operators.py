"""What is measured of the operators between attention and the loss, case by case.

Four operators of a language model's training step, each with its gradient:
dropout whose mask is never stored, the residual's addition with RMS norm
(and an output in 8 bits), matrix products grouped by expert, and the log
probabilities of given tokens with entropy and top alternatives. ``run``
computes them in plain torch operations (``own`` false) or through the
package's entry points (``own`` true). Sizes follow the repository's own
workloads: the 1000 x 256 embedding of its tiny workload, the vocabulary of
151936 and the width of 2048 of its large one, and the 1024- and 2048-wide
action experts with their four times wider hidden layers.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ---- the cases ----

def listed():
    return [
        # one position of an answer with its alternatives, as a policy's rollout asks for it
        {"name": "logprob_one", "op": "token_logprobs", "tokens": 1, "vocab": 151936, "dtype": "bf16", "top": 8},
        # a whole batch of answers, with the alternatives that a distillation or a report keeps
        {"name": "logprob_batch", "op": "token_logprobs", "tokens": 4093, "vocab": 151936, "dtype": "bf16", "top": 20},
        # the tiny workload's loss, in fp32
        {"name": "logprob_grad_tiny", "op": "token_logprobs_backward", "tokens": 61, "vocab": 1000, "dtype": "fp32"},
        # the gradient of a whole batch's loss with an entropy term
        {"name": "logprob_grad_batch", "op": "token_logprobs_backward", "tokens": 4093, "vocab": 151936,
         "dtype": "bf16"},
        # one chunk of 50 action tokens on its way to a product in 8 bits
        {"name": "norm_chunk", "op": "residual_norm", "tokens": 50, "width": 1024, "dtype": "bf16", "stream": "bf16",
         "p": 0.0, "eight_bit": True},
        # the backbone's residual stream for a whole batch, the branch with dropout
        {"name": "norm_batch", "op": "residual_norm", "tokens": 32749, "width": 2048, "dtype": "bf16",
         "stream": "bf16", "p": 0.1, "eight_bit": False},
        # its gradient
        {"name": "norm_grad_batch", "op": "residual_norm_backward", "tokens": 32749, "width": 2048, "dtype": "bf16",
         "stream": "bf16", "p": 0.1},
        # dropout of the tiny workload's activations, in fp32
        {"name": "dropout_tiny", "op": "dropout", "tokens": 777, "width": 256, "dtype": "fp32", "p": 0.1},
        # dropout of a hidden layer of the 2048-wide expert for a batch
        {"name": "dropout_batch", "op": "dropout", "tokens": 16381, "width": 8192, "dtype": "bf16", "p": 0.1},
        # one chunk of action tokens over eight experts
        {"name": "expert_chunk", "op": "expert_matmul", "lengths": "7,0,13,1,9,4,0,16", "inner": 1024, "outer": 4096},
        # a batch routed to eight experts, one of them hardly used
        {"name": "expert_batch", "op": "expert_matmul", "lengths": "2048,1777,3011,130,2900,1,2593,3900",
         "inner": 2048, "outer": 8192},
        # the gradients of the same layer
        {"name": "expert_grad_batch", "op": "expert_matmul_backward",
         "lengths": "2048,1777,3011,130,2900,1,2593,3900", "inner": 2048, "outer": 8192, "grad": "bf16"},
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["token_logprobs", "token_logprobs_backward", "residual_norm", "residual_norm_backward",
                     "dropout", "expert_matmul", "expert_matmul_backward"])
    if op.startswith("token_logprobs"):
        vocab, dtype = log_int(rng, 1000, 151936), rng.choice(["bf16", "bf16", "fp32"])
        most = 3 * 10 ** 8 if dtype == "fp32" else 6 * 10 ** 8
        case = {"op": op, "tokens": log_int(rng, 1, min(8192, most // vocab)), "vocab": vocab, "dtype": dtype}
        return {**case, "top": rng.choice([0, 1, 5, 8, 20, 32])} if op == "token_logprobs" else case
    if op.startswith("residual_norm"):
        width = 8 * log_int(rng, 16, 1024)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        stream = "fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"])
        most = 3 * 10 ** 7 if stream == "fp32" else 6 * 10 ** 7
        case = {"op": op, "tokens": log_int(rng, 1, min(32749, most // width)), "width": width, "dtype": dtype,
                "stream": stream, "p": rng.choice([0.0, 0.1, 0.5])}
        return {**case, "eight_bit": rng.random() < 0.5} if op == "residual_norm" else case
    if op == "dropout":
        width, dtype = log_int(rng, 100, 8192), rng.choice(["bf16", "bf16", "fp32"])
        most = 6 * 10 ** 7 if dtype == "fp32" else 12 * 10 ** 7
        return {"op": op, "tokens": log_int(rng, 1, min(32749, most // width)), "width": width, "dtype": dtype,
                "p": rng.choice([0.05, 0.1, 0.3, 0.5])}
    total, experts = log_int(rng, 1, 8192), rng.choice([1, 4, 8, 8, 16, 40, 64])
    cuts = sorted(rng.randint(0, total) for _ in range(experts - 1))
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    case = {"op": op, "lengths": ",".join(str(n) for n in lengths), "inner": 8 * log_int(rng, 16, 256),
            "outer": 8 * log_int(rng, 16, 512)}
    return {**case, "grad": rng.choice(["bf16", "fp32"])} if op == "expert_matmul_backward" else case


def lengths_of(case):
    return [int(n) for n in case["lengths"].split(",")]


# ---- inputs ----

PAD = 1 / 512  # of the vocabulary's columns, the last, belong to no token: their logits are masked


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    op = case["op"]
    s = {"op": op}
    if op.startswith("token_logprobs"):
        n, v = case["tokens"], case["vocab"]
        # most tokens are unlikely, a few stand out, and the one that followed is often among these
        logits = normal(n, v, std=2.0, dtype=torch.float32)
        likely = torch.randint(0, v - int(v * PAD), (n, 4), generator=gen, device="cuda")
        logits.scatter_(1, likely, 12 + normal(n, 4, std=2.0, dtype=torch.float32))
        logits[:, v - int(v * PAD):] = -math.inf
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        ids = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.7, likely[:, 0],
                          torch.randint(0, v - int(v * PAD), (n,), generator=gen, device="cuda"))
        prompt = torch.rand(n, generator=gen, device="cuda") < 0.1  # positions that take no part in the loss
        s["ids"], s["scale"] = ids.masked_fill(prompt, -100), 1 / 0.8
        if op.endswith("backward"):
            s["dlogprobs"] = normal(n, std=1 / n, dtype=torch.float32)
            s["dentropy"] = normal(n, std=0.1 / n, dtype=torch.float32)
            _, s["entropy"], s["lse"] = plain_logprobs(s)
        else:
            s["top"] = case["top"]
    elif op == "dropout":
        s["x"], s["p"] = normal(case["tokens"], case["width"], dtype=DTYPES[case["dtype"]]), case["p"]
    elif op.startswith("residual_norm"):
        n, w, dt, st = case["tokens"], case["width"], DTYPES[case["dtype"]], DTYPES[case["stream"]]
        s["weight"], s["p"] = 1 + normal(w, std=0.1, dtype=torch.float32), case["p"]
        # a residual stream has some channels far above the others
        loud = 1 + 20 * (torch.rand(w, generator=gen, device="cuda") < 0.01)
        s["residual"] = (normal(n, w, std=2.0, dtype=torch.float32) * loud).to(st)
        if op.endswith("backward"):
            s["dy"], s["dres"] = normal(n, w, std=1e-3, dtype=dt), normal(n, w, std=1e-3, dtype=st)
        else:
            s["x"], s["eight_bit"] = normal(n, w, dtype=dt), case["eight_bit"]
    else:
        lengths, k, n = lengths_of(case), case["inner"], case["outer"]
        s["x"] = normal(sum(lengths), k)
        s["weight"] = normal(len(lengths), n, k, std=0.02)
        s["lengths"] = lengths
        s["offsets"] = torch.tensor(np.cumsum([0] + lengths), device="cuda", dtype=torch.int32)
        if op.endswith("backward"):
            s["dout"] = normal(sum(lengths), n, std=1e-3)
            # the gradient buffer that the optimizer has registered
            s["grad"] = torch.empty(len(lengths), n, k, device="cuda", dtype=DTYPES[case["grad"]])
    if "p" in s:
        # the generator's key and step, which a training loop counts up on the GPU
        s["rng"] = torch.randint(0, 2 ** 62, (2,), generator=gen, device="cuda")
        s["site"] = 3
    return s


# ---- the plain forms ----

def plain_mul(c, x):
    """High and low 32 bits of a constant times 32-bit values that int64 holds."""
    p = (x & 0xFFFF) * c
    t = (x >> 16) * c + (p >> 16)
    return t >> 16, (t & 0xFFFF) << 16 | p & 0xFFFF


def plain_keep(s, n):
    """Which of n elements dropout keeps: 16 bits for each from Philox4x32-10 (Salmon and others, 2011). The key is
    the seed; the counter is the group of eight elements, the site and the step."""
    c0 = torch.arange((n + 7) // 8, device="cuda")
    seed, step = s["rng"][0], s["rng"][1]
    c1, c2, c3 = torch.full_like(c0, s["site"]), (step & 0xFFFFFFFF).expand_as(c0), (step >> 32 & 0xFFFFFFFF).expand_as(c0)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF
    for _ in range(10):
        (h0, l0), (h1, l1) = plain_mul(0xD2511F53, c0), plain_mul(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = k0 + 0x9E3779B9 & 0xFFFFFFFF, k1 + 0xBB67AE85 & 0xFFFFFFFF
    words = torch.stack((c0, c1, c2, c3), -1)
    bits = torch.stack((words & 0xFFFF, words >> 16), -1).flatten()[:n]
    return bits >= dropped_of_65536(s)


def dropped_of_65536(s):
    return int(math.floor(s["p"] * 65536 + 0.5))


def plain_dropout(s, x):
    """In fp32."""
    if s["p"] == 0:
        return x.float()
    keep = plain_keep(s, x.numel()).view(x.shape)
    return torch.where(keep, x.float() * (65536 / (65536 - dropped_of_65536(s))), 0)


def plain_residual_norm(s):
    r = s["residual"].float() + plain_dropout(s, s["x"])
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"]
    if not s["eight_bit"]:
        return y.to(s["x"].dtype), r.to(s["residual"].dtype)
    scales = y.abs().amax(-1) / 448
    return (y / scales[:, None]).to(torch.float8_e4m3fn), scales, r.to(s["residual"].dtype)


def plain_residual_norm_backward(s):
    r = s["residual"].float()
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    y, dy = r * rstd, s["dy"].float()
    g = dy * s["weight"]
    dr = s["dres"].float() + rstd * (g - y * (g * y).mean(-1, keepdim=True))
    return plain_dropout(s, dr).to(s["dy"].dtype), dr.to(s["dres"].dtype), (dy * y).sum(0)


def plain_logprobs(s):
    x = s["logits"].float() * s["scale"]
    top = x.amax(-1, keepdim=True)
    x.sub_(top)
    e = torch.exp(x)
    total = e.sum(-1)
    of_mean = e.mul_(x.clamp_(min=-1e30)).sum(-1) / total
    inside = (s["ids"] >= 0) & (s["ids"] < x.shape[1])
    at = x.gather(1, s["ids"].clamp(0, x.shape[1] - 1)[:, None])[:, 0]
    log_total = total.log()
    return torch.where(inside, at - log_total, 0), log_total - of_mean, top[:, 0] + log_total


def plain_top(s, lse):
    """The largest logits, the lowest index first among equal ones, by integers that sort as the pairs do."""
    x = s["logits"].float() + 0.0
    bits = x.view(torch.int32)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    v = x.shape[1]
    key = bits * 2 ** 32 + (v - 1 - torch.arange(v, device="cuda"))
    ids = v - 1 - (key.topk(s["top"], dim=-1).values & 0xFFFFFFFF)
    return x.gather(1, ids) * s["scale"] - lse[:, None], ids


def plain_logprobs_backward(s):
    logp = (s["logits"].float() * s["scale"] - s["lse"][:, None]).clamp_(min=-1e30)
    p = torch.exp(logp)
    d = p * (-s["dlogprobs"] * inside_of(s))[:, None] - p * s["dentropy"][:, None] * (logp + s["entropy"][:, None])
    d.scatter_add_(1, s["ids"].clamp(min=0)[:, None], (s["dlogprobs"] * inside_of(s))[:, None])
    return (d * s["scale"]).to(s["logits"].dtype)


def inside_of(s):
    return (s["ids"] >= 0) & (s["ids"] < s["logits"].shape[1])


def plain_expert_matmul(s):
    parts = zip(s["x"].float().split(s["lengths"]), s["weight"].float())
    return torch.cat([a @ w.T for a, w in parts]).to(s["x"].dtype)


def plain_expert_matmul_backward(s):
    x, dout, w = s["x"].float().split(s["lengths"]), s["dout"].float().split(s["lengths"]), s["weight"].float()
    dx = torch.cat([d @ b for d, b in zip(dout, w)]).to(s["x"].dtype)
    return dx, s["grad"].copy_(torch.stack([d.T @ a for d, a in zip(dout, x)]))


def run_plain(s):
    op = s["op"]
    if op == "token_logprobs":
        logprobs, entropy, lse = plain_logprobs(s)
        return (logprobs, entropy, lse, *plain_top(s, lse)) if s["top"] else (logprobs, entropy, lse)
    if op == "token_logprobs_backward":
        return plain_logprobs_backward(s)
    if op == "dropout":
        return plain_dropout(s, s["x"]).to(s["x"].dtype)
    if op == "residual_norm":
        return plain_residual_norm(s)
    if op == "residual_norm_backward":
        return plain_residual_norm_backward(s)
    return plain_expert_matmul(s) if op == "expert_matmul" else plain_expert_matmul_backward(s)


def run(s):
    if not own:
        return run_plain(s)
    from muon_adamw_hybrid_grad_gb300 import ops

    op = s["op"]
    if op == "token_logprobs":
        got = ops.token_logprobs(s["logits"], s["ids"], scale=s["scale"], top=s["top"])
        return got if s["top"] else got[:3]
    if op == "token_logprobs_backward":
        return ops.token_logprobs_backward(s["dlogprobs"], s["dentropy"], s["logits"], s["ids"], s["entropy"],
                                           s["lse"], scale=s["scale"])
    if op == "dropout":
        return ops.dropout(s["x"], s["p"], s["rng"], site=s["site"])
    if op == "residual_norm":
        return ops.residual_norm(s["x"], s["residual"], s["weight"], eps=EPS, p=s["p"], rng=s["rng"], site=s["site"],
                                 eight_bit=s["eight_bit"])
    if op == "residual_norm_backward":
        return ops.residual_norm_backward(s["dy"], s["dres"], s["residual"], s["weight"], eps=EPS, p=s["p"],
                                          rng=s["rng"], site=s["site"])
    if op == "expert_matmul":
        return ops.expert_matmul(s["x"], s["weight"], s["offsets"])
    return ops.expert_matmul_backward(s["dout"], s["x"], s["weight"], s["offsets"], s["grad"])


# ---- what a pass cannot do without ----

def work(case):
    op = case["op"]
    size = {"fp32": 4, "bf16": 2}
    if op.startswith("token_logprobs"):
        n, v, b = case["tokens"], case["vocab"], size[case["dtype"]]
        if op.endswith("backward"):
            # logits, ids and four values a row in, the logits' gradient out
            return {"bytes": 2 * n * v * b + n * 24, "flops": 8 * n * v}
        return {"bytes": n * v * b + n * (20 + 12 * case["top"]), "flops": 6 * n * v}
    if op == "dropout":
        n = case["tokens"] * case["width"]
        return {"bytes": 2 * n * size[case["dtype"]], "flops": n}
    if op.startswith("residual_norm"):
        n, w = case["tokens"], case["width"]
        dt, st = size[case["dtype"]], size[case["stream"]]
        if op.endswith("backward"):
            # dy, dres and the stream in; both gradients out, unless without dropout they are one
            outs = st if case["p"] == 0 and dt == st else dt + st
            return {"bytes": n * w * (dt + 2 * st + outs) + 8 * w, "flops": 12 * n * w}
        y = n * (w + 4) if case["eight_bit"] else n * w * dt
        return {"bytes": n * w * (dt + 2 * st) + y + 4 * w, "flops": 6 * n * w}
    lengths, k, n = lengths_of(case), case["inner"], case["outer"]
    t, used = sum(lengths), sum(x > 0 for x in lengths)
    if op == "expert_matmul":
        return {"bytes": 2 * (t * (k + n) + used * n * k), "flops": 2 * t * n * k}
    # x, dout and the weights that are used in, dx and every expert's gradient out; two products
    return {"bytes": 2 * (t * (2 * k + n) + used * n * k) + len(lengths) * n * k * size[case["grad"]],
            "flops": 4 * t * n * k}


# ---- the definitions in 64 bits ----

def exact_keep(s, n):
    """The generator over numpy's unsigned integers."""
    low = np.uint64(0xFFFFFFFF)
    c = np.zeros((4, (n + 7) // 8), np.uint64)
    seed, step = (int(x) for x in s["rng"].cpu())
    c[0] = np.arange(c.shape[1])
    c[1], c[2], c[3] = s["site"], step & 0xFFFFFFFF, step >> 32
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = np.stack((b >> np.uint64(32) ^ c[1] ^ np.uint64(key[0]), b & low,
                      a >> np.uint64(32) ^ c[3] ^ np.uint64(key[1]), a & low))
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    halves = np.ascontiguousarray(c.T.astype("<u4")).view("<u2").reshape(-1)[:n]
    return torch.from_numpy(halves.astype(np.int32)).cuda() >= round(s["p"] * 65536)


def exact_dropout(s, x):
    if s["p"] == 0:
        return x
    kept = exact_keep(s, x.numel()).view_as(x).double()
    return x * kept / (1 - round(s["p"] * 65536) / 65536)


def to_e4m3(y):
    """The nearest values of 3 bits of fraction, an even last bit where two are as near, subnormal below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        return exact_dropout(s, s["x"].double())
    if op == "residual_norm":
        r = s["residual"].double() + exact_dropout(s, s["x"].double())
        y = r / torch.sqrt(r.square().sum(-1, keepdim=True) / r.shape[-1] + EPS) * s["weight"].double()
        if not s["eight_bit"]:
            return y, r
        scales = y.abs().max(-1).values / 448
        return to_e4m3(y / scales[:, None]), scales, r
    if op == "residual_norm_backward":
        r, w = s["residual"].double().requires_grad_(), s["weight"].double().requires_grad_()
        y = r / torch.sqrt(r.square().sum(-1, keepdim=True) / r.shape[-1] + EPS) * w
        dr, dw = torch.autograd.grad((y, r * 1), (r, w), (s["dy"].double(), s["dres"].double()))
        return exact_dropout(s, dr), dr, dw
    if op.startswith("token_logprobs"):
        got = [exact_logprobs(s, rows) for rows in torch.arange(case["tokens"], device="cuda").split(512)]
        got = [torch.cat(x) if x[0] is not None else None for x in zip(*got)]
        return got[0] if op.endswith("backward") else tuple(got)
    x, w = s["x"].double(), s["weight"].double()
    expert = torch.repeat_interleave(torch.tensor(s["lengths"])).tolist()
    bounds = [0, *np.cumsum(s["lengths"]).tolist()]
    if op == "expert_matmul":
        out = x.new_empty(len(expert), case["outer"])
        for e in set(expert):
            out[bounds[e]:bounds[e + 1]] = torch.einsum("tk,nk->tn", x[bounds[e]:bounds[e + 1]], w[e])
        return out
    dx, dw, dout = torch.zeros_like(x), torch.zeros_like(w), s["dout"].double()
    for e in set(expert):
        rows = slice(bounds[e], bounds[e + 1])
        dx[rows] = torch.einsum("tn,nk->tk", dout[rows], w[e])
        dw[e] = torch.einsum("tn,tk->nk", dout[rows], x[rows])
    return dx, dw


def exact_logprobs(s, rows):
    back = s["op"].endswith("backward")
    x = s["logits"][rows].double().requires_grad_(back)
    logp = torch.log_softmax(x * s["scale"], -1)
    entropy = -(logp.exp() * logp.masked_fill(logp == -math.inf, 0)).sum(-1)
    ids = s["ids"][rows]
    chosen = torch.cat((logp, logp.new_zeros(len(rows), 1)), 1)[torch.arange(len(rows)), ids.clamp(min=-1)]
    if back:
        return torch.autograd.grad((chosen, entropy), x, (s["dlogprobs"][rows].double(), s["dentropy"][rows].double()))
    lse = torch.logsumexp(x * s["scale"], -1)
    if not s["top"]:
        return chosen, entropy, lse
    return chosen, entropy, lse, logp.topk(s["top"], -1).values, None
