"""The measured cases of gradient clipping and of drafted tokens' verification: the
norm of many gradient tensors, their clipping, the sharded step with clipping,
and the accepted tokens of a draft with the token drawn after them.

``run`` makes one pass of a case: with ``own`` false in the operators' plain
form (elementary torch operations), with ``own`` true through the library's
entry points.  Parameter lists are those of this repository's workloads (the
three-layer toy, GPT-2-small, the ragged list, the 1.3B decoder), vocabularies
those of its language models (50257, 32000).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}
HP = dict(lr=5e-5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)

TOY = [784 * 1024, 1024, 1024 * 256, 256, 256 * 10, 10]


def _gpt(layers, d, vocab, ctx):
    block = [d, d, d * 3 * d, 3 * d, d * d, d, d, d, d * 4 * d, 4 * d, 4 * d * d, d]
    return [vocab * d, ctx * d] + block * layers + [d, d]


def _ragged(count, low, high, seed):
    """Sizes spread over their logarithm, odd ones and single elements among them."""
    r = torch.rand(count, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    return [max(1, int(v)) for v in torch.exp(math.log(low) + r * math.log(high / low)).tolist()]


def _numels(c):
    if c["list"] == "toy":
        return TOY
    if c["list"] == "gpt":
        return _gpt(c["layers"], c["dim"], c["vocab"], c["ctx"])
    return _ragged(c["count"], c["low"], c["high"], c["sizes"])


def listed():
    small = dict(list="gpt", layers=12, dim=768, vocab=50257, ctx=1024)
    return [
        # The norm of a small model's gradients: latency alone.
        dict(name="norm toy", op="norm", list="toy", dtype="bf16", tensor_norms=True),
        # Gradients of GPT-2-small accumulated in 32 bits, each tensor's norm beside the total.
        dict(name="norm gpt2", op="norm", dtype="f32", tensor_norms=True, **small),
        # Two thousand tensors of 1 to 4e6 elements.
        dict(name="norm ragged", op="norm", list="ragged", count=2000, low=1, high=4_000_000, sizes=5,
             dtype="bf16", tensor_norms=False),
        # Clipping of the small model's gradients.
        dict(name="clip toy", op="clip", list="toy", dtype="bf16", out="bf16", tensor_norms=False),
        # GPT-2-small's 32-bit gradients, clipped into the rank's bf16 gradients.
        dict(name="clip gpt2", op="clip", dtype="f32", out="bf16", tensor_norms=True, **small),
        # The toy's sharded step with clipping, two ranks and five persistent tensors.
        dict(name="step toy", op="step", psi=TOY[0] + TOY[2], psi_s=1024 + 256 + 2560 + 10, nd=2),
        # GPT-2-small over seven ranks: shards that start at odd elements.
        dict(name="step gpt2", op="step", psi=124_318_464, psi_s=121_344, nd=7),
        # The 1.3B decoder over eight ranks.
        dict(name="step decoder", op="step", psi=1_315_080_192, psi_s=643_072, nd=8),
        # One sequence decoding with four drafted tokens.
        dict(name="verify one", op="verify", n=1, k=4, vocab=50257, dtype="bf16", ids="i64",
             draft="logits", masked=0.0),
        # Sampling without a draft for a batch, a mask over some of the rows, 32-bit logits.
        dict(name="verify sample", op="verify", n=128, k=0, vocab=32000, dtype="f32", ids="i32",
             draft="none", masked=0.3),
        # Tokens copied from the prompt (no draft probabilities), ten for each of 48 sequences.
        dict(name="verify lookup", op="verify", n=48, k=10, vocab=50257, dtype="bf16", ids="i32",
             draft="none", masked=0.0),
        # Rollouts of a policy: 512 sequences with five tokens from a draft model.
        dict(name="verify rollout", op="verify", n=512, k=5, vocab=50257, dtype="bf16", ids="i64",
             draft="logits", masked=0.0),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "step", "verify", "verify"])
    if op in ("norm", "clip"):
        c = dict(op=op, dtype=rng.choice(["bf16", "f32"]), tensor_norms=rng.random() < 0.5)
        if op == "clip":
            c["out"] = rng.choice([c["dtype"], "bf16", "f32"])
        if rng.random() < 0.3:
            d = 64 * rng.randint(2, 12)
            c.update(list="gpt", layers=rng.randint(1, 12), dim=d, vocab=_logu(rng, 1000, 50257), ctx=_logu(rng, 64, 1024))
        else:
            low = _logu(rng, 1, 5000)
            c.update(list="ragged", count=_logu(rng, 1, 2500), low=low, sizes=rng.randint(0, 10 ** 6))
            c["high"] = max(low + 1, min(_logu(rng, 1000, 20_000_000), 200_000_000 // c["count"]))
        return c
    if op == "step":
        nd = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 16])
        return dict(op=op, psi=_logu(rng, 100_000, 600_000_000 // nd), psi_s=_logu(rng, 1, 99_999), nd=nd)
    vocab = min(100_000, _logu(rng, 1000, 110_000))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    k = rng.choice([0, 1, 2, 3, 4, 5, 7, 10])
    n = max(1, min(_logu(rng, 1, 512), 512 * 11 * 50257 * 2 // ((2 * k + 3) * vocab * BYTES[dtype])))
    return dict(op=op, n=n, k=k, vocab=vocab, dtype=dtype, ids=rng.choice(["i32", "i64"]),
                draft=rng.choice(["logits", "logits", "none"]) if k else "none",
                masked=rng.choice([0.0, 0.0, 0.3]))


# Share of drafted tokens that are accepted with the inputs made here: a draft
# model's, and a single proposed token's.
ACCEPTED = {"logits": 0.77, "none": 0.65}


def work(case):
    c = case
    if c["op"] in ("norm", "clip"):
        n = sum(_numels(c))
        b = n * BYTES[c["dtype"]]
        if c["op"] == "clip":
            b += n * BYTES[c["out"]]
        return dict(bytes=b, flops=n * (2 + (c["op"] == "clip")))
    if c["op"] == "step":
        # the norm and the update both need every gradient, which are read once
        return dict(bytes=c["psi"] * (2 * c["nd"] + 28) + c["psi_s"] * (2 * c["nd"] + 26),
                    flops=(c["psi"] + c["psi_s"]) * (c["nd"] + 18))
    # rows up to the first refusal, and the noise
    a = ACCEPTED[c["draft"]]
    k, V = c["k"], c["vocab"]
    pairs = sum(a ** j for j in range(k))
    rows = pairs * (2 if c["draft"] == "logits" else 1) + a ** k
    return dict(bytes=c["n"] * V * (rows * BYTES[c["dtype"]] + 4), flops=c["n"] * V * (5 * rows + 6))


def _gen(seed):
    return torch.Generator("cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)


def prepare(case, seed):
    return dict(norm=_prepare_list, clip=_prepare_list, step=_prepare_step,
                verify=_prepare_verify)[case["op"]](case, _gen(seed), seed)


def _prepare_list(c, g, seed):
    numels = _numels(c)
    # the sizes differ from tensor to tensor: layers have gradients of other scales
    flat = torch.randn(sum(numels), generator=g, device="cuda")
    scale = torch.exp(torch.randn(len(numels), generator=g, device="cuda") - 6.0)
    flat *= torch.repeat_interleave(scale, torch.tensor(numels, device="cuda"))
    flat = flat.to(DT[c["dtype"]])
    f32 = dict(device="cuda", dtype=torch.float32)
    s = dict(case=c, flat=flat, numels=numels, tensors=list(flat.split(numels)), max_norm=1.0,
             norm=torch.empty(1, **f32), coef=torch.empty(1, **f32))
    s["tensor_norms"] = torch.empty(len(numels), **f32) if c["tensor_norms"] else None
    if c["op"] == "clip":
        s["max_norm"] = 0.25 * math.sqrt(sum(numels)) * math.exp(-6.0)
        s["out_flat"] = torch.empty(sum(numels), device="cuda", dtype=DT[c["out"]])
        s["out"] = list(s["out_flat"].split(numels))
    return s


def _rows(n, cols, dtype, fill=None):
    """n rows of cols elements, each on a 16-byte boundary."""
    x = torch.zeros(n, (cols + 7) // 8 * 8, device="cuda", dtype=dtype)
    if fill is not None:
        x[:, :cols] = fill
    return x


def _prepare_step(c, g, seed):
    nd, psi, ps = c["nd"], c["psi"], c["psi_s"]
    S = -(-psi // nd)
    pad = S * nd
    rand = lambda *a: torch.randn(*a, generator=g, device="cuda")  # noqa: E731
    # each rank's gradients: the flat ones, then the persistent group's
    at = (pad + 7) // 8 * 8
    grads = torch.empty(nd, (at + ps + 7) // 8 * 8, device="cuda", dtype=torch.bfloat16)
    for q in range(nd):
        for a in range(0, grads.shape[1], 1 << 28):
            b = min(grads.shape[1], a + (1 << 28))
            grads[q, a:b] = rand(b - a) * 1e-3
    grads[:, psi:at] = 0
    s = dict(case=c, S=S, pad=pad, at=at, grads=grads, t=3)
    s["max_norm"] = 0.4e-3 / math.sqrt(nd) * math.sqrt(psi + ps)
    for name, scale in (("master", 0.02), ("m", 1e-4), ("v", 1e-7)):
        x = s[name] = _rows(nd, S, torch.float32)
        for r in range(nd):
            x[r, :S] = rand(S) * scale if name != "v" else torch.rand(S, generator=g, device="cuda") * scale
            x[r, max(0, min(S, psi - r * S)):] = 0
        p = s["p" + name] = rand(ps) * scale
        if name == "v":
            p.abs_()
    s["sparam"] = _rows(nd, S, torch.bfloat16)
    s["full"] = torch.zeros(pad, device="cuda", dtype=torch.bfloat16)
    s["pparam"] = torch.zeros(ps, device="cuda", dtype=torch.bfloat16)
    s["norm"] = torch.empty(1, device="cuda")
    return s


def _prepare_verify(c, g, seed):
    n, k, V = c["n"], c["k"], c["vocab"]
    dt = DT[c["dtype"]]
    dev = dict(generator=g, device="cuda")
    x = torch.empty(n, k + 1, V, device="cuda", dtype=dt)
    y = torch.empty(n, k, V, device="cuda", dtype=dt) if c["draft"] == "logits" else None
    ids = torch.empty(n, k, device="cuda", dtype=torch.int64)
    for a in range(0, n, 64):
        b = min(n, a + 64)
        z = torch.randn(b - a, k + 1, V, **dev) * 2.5
        top = torch.randint(0, V, (b - a, k + 1, 4), **dev)  # a few likely tokens
        z.scatter_add_(2, top, 4.0 + 6.0 * torch.rand(b - a, k + 1, 4, **dev))
        x[a:b] = z
        if k:
            w = z[:, :k] + 0.6 * torch.randn(b - a, k, V, **dev)
            if y is not None:
                y[a:b] = w
                w = y[a:b].float()
            if y is not None:  # drawn from the draft
                ids[a:b] = (w - torch.log(torch.empty_like(w).exponential_(generator=g))).argmax(2)
            else:  # copied tokens: often right, and then the target is nearly certain
                ids[a:b] = w.argmax(2)
                sure = 8.0 * (torch.rand(b - a, k, 1, **dev) < 0.6)
                z[:, :k].scatter_add_(2, ids[a:b, :, None], sure)
                x[a:b] = z
    scale = 1.0 if seed % 2 else 1.25
    if c["masked"]:  # rows under a mask keep about 40 tokens, a few of them none
        for a in range(0, n, 64):
            b = min(n, a + 64)
            r = torch.rand(b - a, k + 1, 1, **dev)
            keep = torch.rand(b - a, k + 1, V, **dev) < torch.where(r < 0.05 * c["masked"], 0.0, 40.0 / V)
            x[a:b].masked_fill_((r < c["masked"]) & ~keep, float("-inf"))
    if n > 4 and k:  # shorter drafts
        length = torch.randint(0, k + 1, (n, 1), **dev)
        short = torch.rand(n, 1, **dev) < 0.1
        ids.masked_fill_(short & (torch.arange(k, device="cuda") >= length), -1)
    s = dict(case=c, x=x, y=y, ids=ids.to(torch.int32 if c["ids"] == "i32" else torch.int64),
             scale=scale, draft_scale=scale)
    s["u"] = torch.rand(n, k, **dev)
    s["noise"] = torch.empty(n, V, device="cuda").exponential_(generator=g)
    s["accepted"] = torch.empty(n, device="cuda", dtype=torch.int32)
    s["tokens"] = torch.empty(n, k + 1, device="cuda", dtype=torch.int32)
    s["logprobs"] = torch.empty(n, k + 1, device="cuda", dtype=torch.float32)
    return s


# ------------------------------------------------------------- plain form

def _clip_coef(norm, max_norm):
    return torch.clamp(max_norm / (norm + 1e-6), max=1.0)


def _list_out(s):
    r = dict(norm=s["norm"], coef=s["coef"])
    if s["tensor_norms"] is not None:
        r["tensor_norms"] = s["tensor_norms"]
    if s["case"]["op"] == "clip":
        r["out"] = s["out_flat"]
    return r


def _plain_list(s):
    # one pass over all tensors where they need not be told apart
    if s["tensor_norms"] is None:
        squares = s["flat"].float().square().sum(dtype=torch.float64)
    else:
        squares = torch.stack([x.float().square().sum(dtype=torch.float64) for x in s["tensors"]])
        s["tensor_norms"].copy_(squares.sqrt())
    norm = squares.sum().sqrt()
    s["norm"].copy_(norm)
    s["coef"].copy_(_clip_coef(norm, s["max_norm"]))
    if s["case"]["op"] == "clip":
        s["out_flat"].copy_(s["flat"].float() * s["coef"])
    return _list_out(s)


def _scalars(t):
    b1, b2 = HP["beta1"] ** t, HP["beta2"] ** t
    return (1.0 - HP["lr"] * HP["weight_decay"], HP["lr"] / (1.0 - b1), 1.0 / math.sqrt(1.0 - b2))


def _plain_adamw(p, m, v, g, t):
    decay, step, inv = _scalars(t)
    p.mul_(decay)
    m.mul_(HP["beta1"]).add_(g * (1.0 - HP["beta1"]))
    v.mul_(HP["beta2"]).add_(g * g * (1.0 - HP["beta2"]))
    p.sub_(m / (v.sqrt() * inv + HP["eps"]) * step)


STEP_OUT = ("norm", "master", "m", "v", "sparam", "full", "pmaster", "pm", "pv", "pparam")


def _plain_step(s):
    c, S, nd = s["case"], s["S"], s["case"]["nd"]
    g = s["grads"][0].float()
    for q in range(1, nd):
        g += s["grads"][q]
    g *= 1.0 / nd
    flat, extra = g[:s["pad"]], g[s["at"]:s["at"] + c["psi_s"]]
    norm = (flat.square().sum(dtype=torch.float64) + extra.square().sum(dtype=torch.float64)).sqrt()
    s["norm"].copy_(norm)
    g *= _clip_coef(norm, s["max_norm"]).float()
    for r in range(nd):
        p = s["master"][r, :S]
        _plain_adamw(p, s["m"][r, :S], s["v"][r, :S], flat[r * S:(r + 1) * S], s["t"])
        s["sparam"][r, :S] = p
        s["full"][r * S:(r + 1) * S] = p
    _plain_adamw(s["pmaster"], s["pm"], s["pv"], extra, s["t"])
    s["pparam"].copy_(s["pmaster"])
    return {k: s[k] for k in STEP_OUT}


def _log_softmax(z):
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, torch.zeros_like(m), m)
    return z - m - torch.log(torch.exp(z - m).sum(-1, keepdim=True))


def _plain_verify(s):
    # 64 bits: an accepted token, or the winner of the draw, may hang on the last digit
    n, k, V = s["x"].shape[0], s["x"].shape[1] - 1, s["x"].shape[2]
    logp = _log_softmax(s["x"].double() * s["scale"])
    logp = torch.where(torch.isnan(logp), -torch.inf, logp)  # rows without any token
    ids = s["ids"].long()
    ok = (ids >= 0) & (ids < V)
    at = torch.where(ok, ids, 0)[..., None]
    logq = None
    if k:
        lp = logp[:, :k].gather(2, at)[..., 0]
        lq = torch.zeros_like(lp)
        if s["y"] is not None:
            logq = _log_softmax(s["y"].double() * s["draft_scale"])
            lq = logq.gather(2, at)[..., 0]
        yes = ok & (torch.log(s["u"].double()) + lq < lp)
        a = torch.cumprod(yes.long(), 1).sum(1)
        length = torch.cumprod(ok.long(), 1).sum(1)
    else:
        a = length = torch.zeros(n, device="cuda", dtype=torch.int64)
    rows = torch.arange(n, device="cuda")
    refused = a < length
    last = logp[rows, a]
    p = torch.exp(last)
    r = p
    if k:
        j = torch.where(refused, a, 0)
        if logq is not None:
            q = torch.exp(logq[rows, j])
        else:
            q = torch.zeros_like(p)
            q[rows, at[rows, j, 0]] = 1.0
        r = torch.where(refused[:, None], p - q, p)
    e = s["noise"].double()
    none = ~((r / e) > 0).any(1, keepdim=True)
    score = torch.where(none, p, r) / e
    best = score.amax(1, keepdim=True)
    col = torch.arange(V, device="cuda")
    token = torch.where(score == best, col, V).amin(1)
    token = torch.where(best[:, 0] > 0, token, -1)
    s["accepted"].copy_(a)
    pos = torch.arange(k + 1, device="cuda")[None]
    d = torch.cat([ids, torch.full((n, 1), -1, device="cuda")], 1)
    s["tokens"].copy_(torch.where(pos < a[:, None], d, torch.where(pos == a[:, None], token[:, None], -1)))
    t = s["tokens"].long()
    lps = logp.gather(2, t.clamp(min=0)[..., None])[..., 0]
    lps = torch.where(t >= 0, lps, torch.where(pos == a[:, None], -torch.inf, 0.0))
    s["logprobs"].copy_(lps)
    return {x: s[x] for x in ("accepted", "tokens", "logprobs")}


PLAIN = dict(norm=_plain_list, clip=_plain_list, step=_plain_step, verify=_plain_verify)


# ------------------------------------------------------- the library's form

def _bytes(n):
    return torch.empty(max(1, n), device="cuda", dtype=torch.uint8)


def _own(s):
    from zero_sharded_optimizer_shard_gb300 import zero3 as Z
    c = s["case"]
    dtype = {"bf16": Z.BF16, "f32": Z.F32}
    stream = torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
    if c["op"] in ("norm", "clip"):
        if "list" not in s:
            s["list"] = Z.TensorList([p(x) for x in s["tensors"]], s["numels"], dtype[c["dtype"]])
            s["ws"] = _bytes(Z.zero3_grad_norm_workspace(s["list"]))
            if c["op"] == "clip":
                s["to"] = Z.TensorList([p(x) for x in s["out"]], s["numels"], dtype[c["out"]])
        Z.zero3_grad_norm(s["list"], s["max_norm"], p(s["tensor_norms"]), 0, p(s["norm"]),
                          p(s["coef"]), p(s["ws"]), s["ws"].numel(), stream)
        if c["op"] == "clip":
            Z.zero3_clip_grads(s["list"], p(s["coef"]), s["to"], stream)
        return _list_out(s)
    if c["op"] == "step":
        nd = c["nd"]
        rows = lambda x: [x[r].data_ptr() for r in range(nd)]  # noqa: E731
        if "plan" not in s:
            s["plan"] = Z.Plan([c["psi"], c["psi_s"]], None, nd, threshold=c["psi_s"] + 1)
            s["hp"] = Z.hparams(**HP)
            s["persist"] = Z.persist_state([x + 2 * s["at"] for x in rows(s["grads"])], p(s["pmaster"]),
                                           p(s["pm"]), p(s["pv"]), p(s["pparam"]))
            s["ptrs"] = [rows(s[x]) for x in ("grads", "master", "m", "v", "sparam")]
            s["ws"] = _bytes(Z.zero3_step_clipped_workspace(s["plan"], 0, s["pad"])[1])
        G, master, m, v, sparam = s["ptrs"]
        Z.zero3_step_clipped(s["plan"], s["hp"], s["t"], G, 0, master, m, v, sparam, p(s["full"]),
                             s["persist"], 0, s["pad"], s["max_norm"], p(s["norm"]), p(s["ws"]),
                             s["ws"].numel(), stream)
        return {x: s[x] for x in STEP_OUT}
    it = Z.I32 if c["ids"] == "i32" else Z.I64
    dt, V = dtype[c["dtype"]], c["vocab"]
    Z.zero3_verify_draft(p(s["x"]), dt, c["n"], c["k"], V, V, p(s["y"]), dt, V, p(s["ids"]), it,
                         s["scale"], s["draft_scale"], p(s["u"]), p(s["noise"]), V,
                         p(s["accepted"]), p(s["tokens"]), p(s["logprobs"]), stream)
    return {x: s[x] for x in ("accepted", "tokens", "logprobs")}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------- 64-bit definition

def _exact_list(s):
    c, sizes = s["case"], torch.tensor(s["numels"], device="cuda")
    owner = torch.repeat_interleave(torch.arange(len(s["numels"]), device="cuda"), sizes)
    total = torch.zeros(len(s["numels"]), device="cuda", dtype=torch.float64)
    total.index_add_(0, owner, s["flat"].double() ** 2)
    del owner
    norm = total.sum().sqrt().reshape(1)
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    r = dict(norm=norm, coef=coef)
    if c["tensor_norms"]:
        r["tensor_norms"] = total.sqrt()
    if c["op"] == "clip":
        r["out"] = s["flat"].double() * coef
    return r


def _exact_step(s):
    c, S, nd = s["case"], s["S"], s["case"]["nd"]
    mean = lambda a, b: s["grads"][:, a:b].double().mean(0)  # noqa: E731
    pieces = [(r * S, (r + 1) * S) for r in range(nd)] + [(s["at"], s["at"] + c["psi_s"])]
    norm = sum(float((mean(a, b) ** 2).sum()) for a, b in pieces) ** 0.5
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    t, b1, b2 = s["t"], HP["beta1"], HP["beta2"]
    out = {k: torch.zeros_like(s[k], dtype=torch.float64) for k in STEP_OUT if k not in ("full", "sparam")}
    out["norm"][0] = norm
    out["full"] = torch.empty(s["pad"], device="cuda", dtype=torch.float64)
    out["sparam"] = torch.zeros_like(s["sparam"], dtype=torch.float64)
    for r, (a, b) in enumerate(pieces):
        g = mean(a, b) * coef
        src = [s[k][r, :S] if r < nd else s["p" + k] for k in ("master", "m", "v")]
        p, m, v = [x.double() for x in src]
        m = m + (1 - b1) * (g - m)
        v = v + (1 - b2) * (g ** 2 - v)
        p = p - HP["lr"] * HP["weight_decay"] * p \
            - HP["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + HP["eps"])
        if r == nd:
            out["pmaster"], out["pm"], out["pv"], out["pparam"] = p, m, v, p
        else:
            out["master"][r, :S], out["m"][r, :S], out["v"][r, :S] = p, m, v
            out["sparam"][r, :S] = p
            out["full"][a:b] = p
    return out


def _exact_verify(s):
    n, k, V = s["case"]["n"], s["case"]["k"], s["case"]["vocab"]
    acc, toks, lps = [], [], []
    for i in range(n):
        P = torch.softmax(s["x"][i].double() * s["scale"], 1)
        logP = torch.log_softmax(s["x"][i].double() * s["scale"], 1)
        empty = torch.isneginf(s["x"][i]).all(1, keepdim=True)
        P, logP = P.masked_fill(empty, 0.0), logP.masked_fill(empty, -math.inf)
        draft, u = s["ids"][i].tolist(), s["u"][i].tolist()
        if s["y"] is not None:
            Q = torch.softmax(s["y"][i].double() * s["draft_scale"], 1)
        a, row = 0, None
        while a < k and 0 <= draft[a] < V:
            q = Q[a] if s["y"] is not None else torch.nn.functional.one_hot(
                torch.tensor(draft[a], device="cuda"), V).double()
            if not u[a] * float(q[draft[a]]) < float(P[a, draft[a]]):
                row = P[a] - q
                break
            a += 1
        e = s["noise"][i].double()
        if row is None or not bool((row / e > 0).any()):
            row = P[a]
        value, where = torch.sort(row / e, descending=True, stable=True)
        token = int(where[0]) if float(value[0]) > 0 else -1
        t = draft[:a] + [token] + [-1] * (k - a)
        acc.append(a)
        toks.append(t)
        lps.append([float(logP[j, t[j]]) if t[j] >= 0 else (-math.inf if j == a else 0.0) for j in range(k + 1)])
    i32 = dict(device="cuda", dtype=torch.int32)
    return dict(accepted=torch.tensor(acc, **i32), tokens=torch.tensor(toks, **i32).reshape(n, k + 1),
                logprobs=torch.tensor(lps, device="cuda", dtype=torch.float64).reshape(n, k + 1))


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_list, clip=_exact_list, step=_exact_step, verify=_exact_verify)[case["op"]](s)
