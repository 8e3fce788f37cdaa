"""The vocabulary operators' measured cases: embedding lookup and its gradient,
log probabilities of given tokens, distillation from a teacher's top logits.

``run`` makes one pass of a case: with ``own`` false in the operators' plain
form (elementary torch operations in 32 bits, rounded once at the end), with
``own`` true through the library's entry points.  Vocabularies and widths are
those of the GPT-2-small, 1.3B-decoder, Llama-7B and two-block lists of this
repository's workloads (50257 with 768 and 2048, 32000 with 4096, 1000), row
counts those of their contexts (1024, 2048) times a batch.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}


def listed():
    return [
        # One decoded token's vector from a width-2048 table: latency alone.
        dict(name="embed token", op="embed", n=1, vocab=50257, dim=2048, dtype="bf16", out="bf16",
             ids="i64", scaled=True),
        # Eight prompts of 2048 tokens through the Llama-7B list's table.
        dict(name="embed prompts", op="embed", n=16384, vocab=32000, dim=4096, dtype="bf16",
             out="bf16", ids="i64", scaled=False),
        # The table's gradient for 8 x 1024 tokens of GPT-2-small: every row of
        # the gradient buffer is written.
        dict(name="embed gradient", op="embed_grad", n=8192, vocab=50257, dim=768, dtype="bf16",
             out="bf16", ids="i64", scaled=False, accumulate=False),
        # A tied table at the 1.3B decoder's width: 16 x 2048 tokens are added
        # to the gradient that the output head has left in the buffer.
        dict(name="embed gradient tied", op="embed_grad", n=32768, vocab=50257, dim=2048,
             dtype="bf16", out="bf16", ids="i64", scaled=True, accumulate=True),
        # A small model with odd sizes and a 32-bit gradient.
        dict(name="embed gradient odd", op="embed_grad", n=3001, vocab=1000, dim=257, dtype="f32",
             out="f32", ids="i32", scaled=False, accumulate=False),
        # Four sequences decoding one token each; the answer lists 20 alternatives.
        dict(name="logprobs decode", op="logprobs", n=4, vocab=50257, dtype="bf16", ids="i64", k=20,
             entropy=True, masked=0.0),
        # The policy's log probabilities and entropies over 8 x 1024 tokens.
        dict(name="logprobs batch", op="logprobs", n=8192, vocab=50257, dtype="bf16", ids="i64",
             k=0, entropy=True, masked=0.0),
        # Scoring with alternatives in 32 bits under masks that forbid tokens
        # (some rows keep a handful, some none), an odd vocabulary.
        dict(name="logprobs masked", op="logprobs", n=1021, vocab=31999, dtype="f32", ids="i32",
             k=5, entropy=True, masked=0.25),
        # The gradient of log probabilities and entropies for that batch.
        dict(name="logprobs gradient", op="logprobs_grad", n=8192, vocab=50257, dtype="bf16",
             ids="i64", entropy=True),
        # Evaluation of a student against stored teacher logits: the loss alone.
        dict(name="distill evaluation", op="distill", n=2047, vocab=32000, dtype="f32",
             ids="i32", teacher=32, grad=False),
        # A distillation step over 8 x 1024 tokens: losses and the logits'
        # gradient in one call.
        dict(name="distill training", op="distill", n=8192, vocab=50257, dtype="bf16", ids="i64",
             teacher=64, grad=True),
        # The same gradient when the rows' weights come after the loss.
        dict(name="distill gradient", op="distill_grad", n=4096, vocab=32000, dtype="bf16",
             ids="i32", teacher=100),
    ]


def _logu(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + (v % 1024 == 0)  # powers of two and their like stay with the listed cases


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "logprobs", "logprobs_grad", "distill", "distill_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    ids = rng.choice(["i32", "i64"])
    vocab = min(50257 * 2, _logu(rng, 1000, 110000))
    c = dict(op=op, vocab=vocab, dtype=dtype, ids=ids)
    if op in ("embed", "embed_grad"):
        c["dim"] = rng.choice([_logu(rng, 64, 4096), 8 * _logu(rng, 8, 380)])
        c["vocab"] = min(vocab, 200_000_000 // c["dim"])
        c["n"] = min(_logu(rng, 1, 65536), (32768 * 4096) // c["dim"])
        c["out"] = rng.choice([dtype, dtype, "f32"])
        c["scaled"] = rng.random() < 0.5
        if op == "embed_grad":
            c["accumulate"] = rng.random() < 0.5
        return c
    c["n"] = max(1, min(_logu(rng, 1, 16384), 8000 * 50257 * 2 // (BYTES[dtype] * vocab)))
    if op == "logprobs":
        c["k"] = rng.choice([0, 0, 1, 5, 20, 64])
        c["entropy"] = rng.random() < 0.6
        c["masked"] = rng.choice([0.0, 0.0, 0.3])
    elif op == "logprobs_grad":
        c["entropy"] = rng.random() < 0.6
    else:
        c["teacher"] = min(_logu(rng, 1, 256), vocab // 4)
        if op == "distill":
            c["grad"] = rng.random() < 0.5
    return c


def _token_weights(vocab):
    """Token frequencies of text: proportional to 1 / (rank + 2.7)."""
    w = 1.0 / (np.arange(vocab) + 2.7)
    return w / w.sum()


def _distinct(n, vocab):
    """Expected number of distinct tokens among n."""
    return float(-np.expm1(n * np.log1p(-_token_weights(vocab))).sum())


def work(case):
    c = case
    n, V = c["n"], c["vocab"]
    e = BYTES[c["dtype"]]
    if c["op"] == "embed":
        d = c["dim"]
        return dict(bytes=_distinct(n, V) * d * e + n * d * BYTES[c["out"]] + n * BYTES[c["ids"]],
                    flops=n * d)
    if c["op"] == "embed_grad":
        d, o = c["dim"], BYTES[c["out"]]
        rows = 2 * _distinct(n, V) if c["accumulate"] else V
        return dict(bytes=n * d * e + rows * d * o + n * BYTES[c["ids"]], flops=2 * n * d)
    if c["op"] == "logprobs":
        return dict(bytes=n * V * e + n * (BYTES[c["ids"]] + 8 + 4 * c["entropy"] + 8 * c["k"]),
                    flops=n * V * (5 + 2 * c["entropy"]))
    if c["op"] == "logprobs_grad":
        return dict(bytes=2 * n * V * e + n * (BYTES[c["ids"]] + 16), flops=n * V * 5)
    K = c["teacher"]
    lists = n * K * (e + BYTES[c["ids"]])
    if c["op"] == "distill":
        return dict(bytes=(1 + c["grad"]) * n * V * e + lists + 12 * n,
                    flops=n * V * (5 + 4 * c["grad"]))
    return dict(bytes=2 * n * V * e + lists + 8 * n, flops=n * V * 4)


def _gen(seed):
    return torch.Generator("cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)


def _tokens(g, n, vocab, ids):
    # summed on the host: a sum whose order varies would move a token now and then
    cdf = torch.from_numpy(np.cumsum(_token_weights(vocab))).cuda()
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = torch.searchsorted(cdf, u).clamp_(max=vocab - 1)
    return t.to(torch.int32 if ids == "i32" else torch.int64)


def _logits(g, n, vocab, dt):
    x = torch.empty(n, vocab, device="cuda", dtype=dt)
    for a in range(0, n, 2048):
        b = min(n, a + 2048)
        x[a:b] = torch.randn(b - a, vocab, generator=g, device="cuda") * 2.5
    return x


def prepare(case, seed):
    c, g = case, _gen(seed)
    n, V = c["n"], c["vocab"]
    dt = DT[c["dtype"]]
    s = dict(case=c)
    if c["op"] in ("embed", "embed_grad"):
        d = c["dim"]
        s["ids"] = _tokens(g, n, V, c["ids"])
        s["scale"] = float(np.float32(math.sqrt(d))) if c["scaled"] else 1.0
        if n > 8:  # padding positions
            s["ids"][torch.randint(0, n, (1 + n // 50,), generator=g, device="cuda")] = -1
        if c["op"] == "embed":
            s["table"] = (torch.randn(V, d, generator=g, device="cuda") * 0.02).to(dt)
            s["out"] = torch.empty(n, d, device="cuda", dtype=DT[c["out"]])
        else:
            s["dout"] = (torch.randn(n, d, generator=g, device="cuda") * 1e-3).to(dt)
            s["grad"] = (torch.randn(V, d, generator=g, device="cuda") * 1e-3).to(DT[c["out"]])
        return s
    x = s["x"] = _logits(g, n, V, dt)
    f32 = dict(device="cuda", dtype=torch.float32)
    if c["op"] in ("logprobs", "logprobs_grad"):
        t = s["targets"] = _tokens(g, n, V, c["ids"])
        at = (torch.arange(n, device="cuda"), t.long())
        x[at] = (x[at].float() + 6.0 * torch.rand(n, generator=g, device="cuda")).to(dt)
        if n > 8:
            t[torch.randint(0, n, (1 + n // 50,), generator=g, device="cuda")] = -100
        if c.get("masked"):  # rows under a mask keep about 40 tokens; some of them none
            r = torch.rand(n, generator=g, device="cuda")
            keep = torch.rand(n, V, generator=g, device="cuda") < 40.0 / V
            keep &= (r > 0.1 * c["masked"])[:, None]
            x.masked_fill_((r < c["masked"])[:, None] & ~keep, float("-inf"))
            del keep
        s["scale"] = 1.0 if seed % 2 else float(np.float32(1 / 0.7))
        if c["op"] == "logprobs":
            s["logprob"], s["lse"] = torch.empty(n, **f32), torch.empty(n, **f32)
            s["ent"] = torch.empty(n, **f32) if c["entropy"] else None
            k = c["k"]
            s["top_ids"] = torch.empty(n, k, device="cuda", dtype=torch.int32) if k else None
            s["top_lp"] = torch.empty(n, k, **f32) if k else None
            return s
        s["lse"], s["ent"] = torch.empty(n, **f32), torch.empty(n, **f32)
        for a in range(0, n, 1024):  # what the forward pass left
            z = x[a:a + 1024].float() * s["scale"]
            lse = torch.logsumexp(z, 1)
            s["lse"][a:a + 1024] = lse
            z -= lse[:, None]
            s["ent"][a:a + 1024] = -(z.exp() * z).sum(1)
        s["dlogprob"] = torch.randn(n, generator=g, **f32)
        s["dent"] = torch.full((n,), 0.01, **f32) if c["entropy"] else None
        s["dx"] = torch.empty_like(x)
        return s
    K = c["teacher"]
    it = torch.int32 if c["ids"] == "i32" else torch.int64
    first = torch.randint(0, V, (n, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, V // K), (n, 1), generator=g, device="cuda")
    k = torch.arange(K, device="cuda")
    tid = (first + step * k) % V  # K distinct tokens
    tl = 14.0 - torch.cumsum(torch.rand(n, K, generator=g, device="cuda") * (12.0 / K), 1)
    near = tl + 0.7 * torch.randn(n, K, generator=g, device="cuda")
    x.scatter_(1, tid, near.to(dt))
    if n > 8:  # shorter lists, and rows without a teacher
        length = torch.where(torch.rand(n, 1, generator=g, device="cuda") < 0.1,
                             torch.randint(0, K + 1, (n, 1), generator=g, device="cuda"), K)
        tid = torch.where(k < length, tid, -1)
    s["tid"], s["tl"] = tid.to(it).contiguous(), tl.to(dt)
    s["scale"] = 1.0 if seed % 2 else 0.5
    s["weight"] = (torch.rand(n, generator=g, device="cuda") > 0.1).float() / n
    s["loss"], s["lse"] = torch.empty(n, **f32), torch.empty(n, **f32)
    if c["op"] == "distill_grad":
        for a in range(0, n, 1024):
            s["lse"][a:a + 1024] = torch.logsumexp(x[a:a + 1024].float() * s["scale"], 1)
    if c["op"] == "distill_grad" or c["grad"]:
        s["dx"] = torch.empty_like(x)
    return s


# ------------------------------------------------------------- plain form

def _stats(z):
    m = z.amax(1, keepdim=True)
    m = torch.where(m == -torch.inf, torch.zeros_like(m), m)
    e = torch.exp(z - m)
    S = e.sum(1, keepdim=True)
    return m, e, S


def _plain_embed(s):
    ids = s["ids"].long()
    ok = (ids >= 0) & (ids < s["table"].shape[0])
    rows = s["table"][torch.where(ok, ids, 0)].float() * s["scale"]
    s["out"].copy_(torch.where(ok[:, None], rows, 0.0))
    return s["out"]


def _plain_embed_grad(s):
    grad = s["grad"]
    V = grad.shape[0]
    ids = s["ids"].long()
    at = torch.where((ids >= 0) & (ids < V), ids, V)
    acc = torch.zeros(V + 1, grad.shape[1], device="cuda", dtype=torch.float32)
    acc.index_add_(0, at, s["dout"].float())
    acc = acc[:V] * s["scale"]
    grad.copy_(grad.float() + acc if s["case"]["accumulate"] else acc)
    return grad


def _plain_logprobs(s):
    c = s["case"]
    z = s["x"].float() * s["scale"]
    m, e, S = _stats(z)
    logS = torch.log(S)
    V = z.shape[1]
    t = s["targets"].long()
    ok = (t >= 0) & (t < V)
    dead = S[:, 0] == 0
    lp = z.gather(1, torch.where(ok, t, 0)[:, None])[:, 0] - m[:, 0] - logS[:, 0]
    lp = torch.where(dead, -torch.inf, lp)
    s["logprob"].copy_(torch.where(ok, lp, 0.0))
    s["lse"].copy_((m + logS)[:, 0])
    if c["entropy"]:
        d = torch.where(e > 0, z - m, 0.0)
        h = logS[:, 0] - (e * d).sum(1) / S[:, 0]
        s["ent"].copy_(torch.where(dead, 0.0, h))
    if c["k"]:
        # distinct keys: the value's bits in order, then the lower index first
        b = (s["x"].float() + 0.0).view(torch.int32).long()
        b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
        key = b * (1 << 32) + (V - 1 - torch.arange(V, device="cuda"))
        top = torch.topk(key, c["k"], dim=1).values
        idx = V - 1 - (top & 0xFFFFFFFF)
        s["top_ids"].copy_(idx)
        tlp = z.gather(1, idx) - m - logS
        s["top_lp"].copy_(torch.where(dead[:, None], -torch.inf, tlp))
    return _logprobs_out(s)


def _logprobs_out(s):
    names = dict(logprob="logprob", lse="lse", entropy="ent", top_ids="top_ids",
                 top_logprobs="top_lp")
    return {k: s[v] for k, v in names.items() if s[v] is not None}


def _plain_logprobs_grad(s):
    x = s["x"]
    n, V = x.shape
    d = x.float() * s["scale"] - s["lse"][:, None]
    p = torch.exp(d)
    t = s["targets"].long()
    ok = (t >= 0) & (t < V)
    g = torch.where(ok, s["dlogprob"], 0.0)
    c = g[:, None].expand(n, V)
    if s["dent"] is not None:
        c = c + s["dent"][:, None] * (d + s["ent"][:, None])
    r = -p * c
    r.scatter_add_(1, torch.where(ok, t, 0)[:, None], g[:, None])
    s["dx"].copy_(r * s["scale"])
    return s["dx"]


def _teacher(s, V):
    tid = s["tid"].long()
    ok = (tid >= 0) & (tid < V) & (s["tl"] > -torch.inf)
    t = torch.where(ok, s["tl"].float() * s["scale"], -torch.inf)
    m, e, S = _stats(t)
    some = S > 0
    q = torch.where(some, e / torch.where(some, S, 1.0), 0.0)
    logq = t - m - torch.log(torch.where(some, S, 1.0))
    return torch.where(ok, tid, 0), q, logq, some[:, 0]


def _plain_distill(s):
    z = s["x"].float() * s["scale"]
    V = z.shape[1]
    m, e, S = _stats(z)
    logS = torch.log(S)
    tid, q, logq, some = _teacher(s, V)
    live = some & (S[:, 0] > 0)
    lp = z.gather(1, tid) - m - logS
    T = 1.0 / s["scale"]
    loss = torch.where(q > 0, q * (logq - lp), 0.0).sum(1) * (T * T)
    s["loss"].copy_(torch.where(live, loss, 0.0))
    s["lse"].copy_((m + logS)[:, 0])
    out = dict(loss=s["loss"], lse=s["lse"])
    if s["case"]["grad"]:
        r = e / S
        r.scatter_add_(1, tid, -q)
        s["dx"].copy_(torch.where(live[:, None], r * (s["weight"] * T)[:, None], 0.0))
        out["dx"] = s["dx"]
    return out


def _plain_distill_grad(s):
    V = s["x"].shape[1]
    r = torch.exp(s["x"].float() * s["scale"] - s["lse"][:, None])
    tid, q, _, some = _teacher(s, V)
    live = some & (s["lse"] > -torch.inf)
    r.scatter_add_(1, tid, -q)
    s["dx"].copy_(torch.where(live[:, None], r * (s["weight"] / s["scale"])[:, None], 0.0))
    return s["dx"]


PLAIN = dict(embed=_plain_embed, embed_grad=_plain_embed_grad, logprobs=_plain_logprobs,
             logprobs_grad=_plain_logprobs_grad, distill=_plain_distill,
             distill_grad=_plain_distill_grad)


# ------------------------------------------------------- the library's form

def _own(s):
    from zero_sharded_optimizer_shard_gb300 import zero3 as Z
    c = s["case"]
    n, V = c["n"], c["vocab"]
    dtype = {"bf16": Z.BF16, "f32": Z.F32}
    it = Z.I32 if c["ids"] == "i32" else Z.I64
    dt = dtype[c["dtype"]]
    stream = torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
    op = c["op"]
    if op == "embed":
        d = c["dim"]
        Z.zero3_embedding_forward(p(s["table"]), dt, V, d, d, p(s["ids"]), it, n, s["scale"],
                                  p(s["out"]), dtype[c["out"]], d, stream)
        return s["out"]
    if op == "embed_grad":
        d = c["dim"]
        if "ws" not in s:
            s["ws"] = torch.empty(Z.zero3_embedding_workspace(n, V, d), device="cuda",
                                  dtype=torch.uint8)
        Z.zero3_embedding_backward(p(s["dout"]), dt, d, p(s["ids"]), it, n, s["scale"],
                                   c["accumulate"], p(s["grad"]), dtype[c["out"]], V, d, d,
                                   p(s["ws"]), s["ws"].numel(), stream)
        return s["grad"]
    if op == "logprobs":
        Z.zero3_token_logprobs(p(s["x"]), dt, n, V, V, p(s["targets"]), it, s["scale"], c["k"],
                               p(s["logprob"]), p(s["lse"]), p(s["ent"]), p(s["top_ids"]),
                               p(s["top_lp"]), stream)
        return _logprobs_out(s)
    if op == "logprobs_grad":
        Z.zero3_token_logprobs_backward(p(s["x"]), dt, n, V, V, p(s["targets"]), it, s["scale"],
                                        p(s["lse"]), p(s["ent"]), p(s["dlogprob"]), p(s["dent"]),
                                        p(s["dx"]), V, stream)
        return s["dx"]
    K = c["teacher"]
    if op == "distill":
        dx = s.get("dx")
        Z.zero3_distill_loss(p(s["x"]), dt, n, V, V, p(s["tl"]), dt, p(s["tid"]), it, K, K,
                             s["scale"], p(s["weight"]), p(s["loss"]), p(s["lse"]), p(dx), V,
                             stream)
        out = dict(loss=s["loss"], lse=s["lse"])
        if dx is not None:
            out["dx"] = dx
        return out
    Z.zero3_distill_backward(p(s["x"]), dt, n, V, V, p(s["tl"]), dt, p(s["tid"]), it, K, K,
                             s["scale"], p(s["lse"]), p(s["weight"]), p(s["dx"]), V, stream)
    return s["dx"]


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------- 64-bit definition

def _exact_teacher(tl, tid, scale, V):
    """Teacher probabilities of one block of rows as a dense [rows, V] matrix,
    with each row's sum of q log q."""
    t = tl.double() * scale
    here = (tid >= 0) & (tid < V) & ~torch.isneginf(t)
    t = t.masked_fill(~here, -1e300)
    q = torch.softmax(t, 1).masked_fill(~here, 0.0)
    dense = torch.zeros(tl.shape[0], V, device="cuda", dtype=torch.float64)
    dense.scatter_add_(1, tid.long().clamp(0, V - 1), q)
    return dense, torch.xlogy(q, q).sum(1), here.any(1)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    a = s["scale"]
    if c["op"] == "embed":
        keep = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
        return torch.nn.functional.embedding(s["ids"].long() * keep, s["table"].double()) * a \
            * keep[:, None]
    if c["op"] == "embed_grad":
        res = s["grad"].double() if c["accumulate"] else torch.zeros_like(s["grad"]).double()
        keep = ((s["ids"] >= 0) & (s["ids"] < c["vocab"])).nonzero()[:, 0]
        return res.index_put_((s["ids"][keep].long(),), s["dout"][keep].double() * a,
                              accumulate=True)
    V = c["vocab"]
    parts = []
    for i in range(0, c["n"], 512):
        z = s["x"][i:i + 512].double() * a
        rows = z.shape[0]
        lse = torch.logsumexp(z, 1)
        none = torch.isneginf(lse)
        if c["op"] in ("logprobs", "logprobs_grad"):
            t = s["targets"][i:i + 512].long()
            hit = torch.arange(V, device="cuda")[None, :] == t[:, None]
            listed_t = hit.any(1)
        if c["op"] == "logprobs":
            logp = (z - lse[:, None]).masked_fill(none[:, None], -math.inf)
            lp = logp.masked_fill(~hit, 0.0).sum(1)
            r = dict(logprob=torch.where(listed_t, lp, 0.0), lse=lse)
            if c["entropy"]:
                r["entropy"] = torch.special.entr(torch.exp(logp)).sum(1)
            if c["k"]:
                v, at = torch.sort(s["x"][i:i + 512].double(), dim=1, descending=True, stable=True)
                r["top_ids"] = at[:, :c["k"]].to(torch.int32)
                r["top_logprobs"] = logp.gather(1, at[:, :c["k"]])
        elif c["op"] == "logprobs_grad":
            lse = s["lse"][i:i + 512].double()
            logp = z - lse[:, None]
            prob = torch.exp(logp)
            g = s["dlogprob"][i:i + 512].double() * listed_t
            r = (hit.double() - prob) * g[:, None]
            if s["dent"] is not None:
                r -= s["dent"][i:i + 512].double()[:, None] * prob \
                    * (logp + s["ent"][i:i + 512].double()[:, None])
            r *= a
        else:
            q, qlogq, some = _exact_teacher(s["tl"][i:i + 512], s["tid"][i:i + 512], a, V)
            if c["op"] == "distill_grad":
                lse = s["lse"][i:i + 512].double()
            logp = z - lse[:, None]
            on = some & ~none
            grad = (torch.exp(logp) - q) * (s["weight"][i:i + 512].double() / a)[:, None] \
                * on[:, None]
            if c["op"] == "distill_grad":
                r = grad
            else:
                cross = torch.where(q > 0, q * logp, 0.0).sum(1)
                r = dict(loss=(qlogq - cross) / (a * a) * on, lse=lse)
                if c["grad"]:
                    r["dx"] = grad
        parts.append(r)
    if isinstance(parts[0], dict):
        return {k: torch.cat([q[k] for q in parts]) for k in parts[0]}
    return torch.cat(parts)
