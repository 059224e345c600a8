"""Cases, inputs and plain forms of the operators around the output matrix: the tied embedding, the gradients'
norm, and the rules that logits are adjusted by before they are scored.

Five operators, each with its cases:

* ``embed``       : ``embedding`` - rows of W [V, d] for given tokens, times a scale.
* ``embed_grad``  : ``embedding_backward`` (into a new dW, or added to the loss's dW) and
  ``differentiable_embedding`` (lookup and gradient through autograd).
* ``clip``        : ``gradient_norm`` and ``clip_gradients`` - the norm over many gradient tensors, and
  the gradients scaled to at most a given norm.
* ``adjust``      : ``adjust_logits`` - penalties for repeated tokens, biases and a mask of allowed tokens.
* ``adjust_grad`` : ``adjust_logits_backward`` - its gradient with respect to the logits.

With t_n a position's token (-1: an empty slot, whose row is 0 and takes no part in the gradient):

    y_n  = s W[t_n],   dW[v] = (dW[v] +) s sum over n with t_n = v of g_n
    norm = sqrt(sum g^2),   c = min(1, max_norm / (norm + 1e-6)),   out = c g

A row's history holds the tokens so far, its first `lengths` entries, of which the first `prompt` were
given and the others generated. With seen_v: v is in the history, and c_v: how often it was generated,

    z1 = z / r if seen_v and z > 0, z r if seen_v, z otherwise
    z' = z1 - f c_v - p [c_v > 0] + (sum of v's biases);   -inf where v is not allowed
    dz = 0 where v is not allowed, otherwise g times dz1/dz

``own`` chooses between the plain form (False) and the package's operators (True).
"""
import math

import torch

own = False

EMPTY = -1
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
ALLOWED = {"few": 0.004, "most": 0.98}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token's embedding, scaled by sqrt(d)
        {"name": "embed 1x2880x201088", "op": "embed", "N": 1, "d": 2880, "V": 201088, "type": "bf16"},
        # the embeddings of a training batch of long texts
        {"name": "embed 65536x2880x201088", "op": "embed", "N": 65536, "d": 2880, "V": 201088, "type": "bf16"},
        # a small student's step in 32 bits, a hidden size that is no multiple of a vector
        {"name": "embed_grad 777x1022x32000", "op": "embed_grad", "what": "new", "N": 777, "d": 1022, "V": 32000,
         "type": "fp32", "out": "fp32"},
        # tied embeddings: added to the output matrix's fp32 gradient
        {"name": "embed_grad 32768x2880x201088 tied", "op": "embed_grad", "what": "add", "N": 32768, "d": 2880,
         "V": 201088, "type": "bf16", "out": "fp32"},
        # lookup and gradient of a 16-bit embedding through autograd
        {"name": "embed_grad 16384x2048x128256 autograd", "op": "embed_grad", "what": "autograd", "N": 16384, "d": 2048,
         "V": 128256, "type": "bf16", "out": "bf16"},
        # gradients of adapters of rank 8 beside frozen weights: many small tensors
        {"name": "clip adapters 4x1024", "op": "clip", "what": "clip", "layers": 4, "d": 1024, "f": 0, "V": 0, "rank": 8,
         "type": "fp32", "out": "fp32", "max_norm": 0.25},
        # a whole student: 16-bit gradients of the layers, the output matrix's in 32, all leaving in 16
        {"name": "clip model 16x2048x128256", "op": "clip", "what": "clip", "layers": 16, "d": 2048, "f": 5632,
         "V": 128256, "rank": 0, "type": "bf16", "out": "bf16", "max_norm": 1.0},
        # one sequence being decoded, in place: no more than its few hundred tokens change
        {"name": "adjust 1x201088 in place", "op": "adjust", "N": 1, "V": 201088, "type": "bf16", "L": 1500, "bias": 8,
         "allowed": "none", "in_place": True},
        # constrained decoding of long conversations: an odd vocabulary in 32 bits, few tokens allowed
        {"name": "adjust 64x50001 few allowed", "op": "adjust", "N": 64, "V": 50001, "type": "fp32", "L": 16384,
         "bias": 50, "allowed": "few", "in_place": False},
        # a chunk of positions of sampled answers, to be scored under the rules they were sampled by
        {"name": "adjust 4096x128256", "op": "adjust", "N": 4096, "V": 128256, "type": "bf16", "L": 1024, "bias": 16,
         "allowed": "most", "in_place": False},
        # gradient for a short answer, half-precision logits of an odd vocabulary
        {"name": "adjust_grad 301x50001", "op": "adjust_grad", "N": 301, "V": 50001, "type": "fp16", "L": 700,
         "allowed": "few", "in_place": False},
        # gradient for a training batch of sampled answers
        {"name": "adjust_grad 4096x128256", "op": "adjust_grad", "N": 4096, "V": 128256, "type": "bf16", "L": 1024,
         "allowed": "most", "in_place": False},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "clip", "adjust", "adjust_grad"])
    c = {"op": op}
    if op in ("embed", "embed_grad"):
        c["type"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        c["V"] = _log_uniform(rng, 1000, 201088)
        c["d"] = 8 * _log_uniform(rng, 8, 360) if rng.random() < 0.75 else _log_uniform(rng, 64, 2880)
        c["N"] = _log_uniform(rng, 1, 65536 * 2 // BYTES[c["type"]])
        if op == "embed_grad":
            c["what"] = rng.choice(["new", "add", "autograd"])
            c["out"] = {"new": rng.choice(["fp32", c["type"]]), "add": "fp32", "autograd": c["type"]}[c["what"]]
    elif op == "clip":
        c["what"] = rng.choice(["norm", "clip", "clip"])
        c["type"] = rng.choice(["bf16", "fp16", "fp32"])
        c["out"] = rng.choice([c["type"], "bf16"])
        c["d"] = _log_uniform(rng, 65, 2048)
        c["layers"] = _log_uniform(rng, 1, 16 if c["type"] != "fp32" else 6)
        c["rank"] = rng.choice([0, 0, 4, 16])
        c["f"] = 0 if c["rank"] else int(c["d"] * rng.uniform(1.5, 2.7))
        c["V"] = 0 if c["rank"] else _log_uniform(rng, 1000, 128256)
        c["max_norm"] = rng.choice([0.5, 1.0, 1e6])  # the last one leaves the gradients as they are
    else:
        c["type"] = rng.choice(["bf16", "fp16", "fp32"])
        c["V"] = _log_uniform(rng, 1000, 201088)
        c["N"] = _log_uniform(rng, 1, min(4096, 4096 * 128256 * 2 // (c["V"] * BYTES[c["type"]])))
        c["L"] = _log_uniform(rng, 1, min(32768, 4096 * 1024 // c["N"]))
        if op == "adjust":
            c["bias"] = rng.choice([0, 1, rng.randint(2, 300)])
        c["allowed"] = rng.choice(["none", "few", "most"])
        c["in_place"] = rng.random() < 0.4
    return c


def _distinct(N, V):
    """How many different tokens N draws of _tokens have, on average."""
    r = torch.arange(V, dtype=torch.float64)
    p = torch.log((r + 2) / (r + 1)) / math.log(V + 1)
    return float((1 - (1 - p) ** N).sum())


def work(case):
    if case["op"] in ("embed", "embed_grad"):
        N, d, e = case["N"], case["d"], BYTES[case["type"]]
        rows = _distinct(N, case["V"])
        if case["op"] == "embed":
            return {"bytes": 4 * N + (rows + N) * d * e, "flops": N * d}
        o = BYTES[case["out"]]
        n = 4 * N + N * d * e + (2 * rows * d * o if case["what"] == "add" else case["V"] * d * o)
        if case["what"] == "autograd":
            n += (rows + N) * d * e
        return {"bytes": n, "flops": 2 * N * d}
    if case["op"] == "clip":
        n = [math.prod(shape) for shape, _ in _shapes(case)]
        b = [BYTES[t] for _, t in _shapes(case)]
        back = 0 if case["what"] == "norm" else sum(n) * BYTES[case["out"]]
        return {"bytes": sum(x * y for x, y in zip(n, b)) + back, "flops": 3 * sum(n)}
    N, V, e = case["N"], case["V"], BYTES[case["type"]]
    L = 0.75 * case["L"]
    n = 4 * N * L + 8 * N * case.get("bias", 0) + (N * V / 8 if case["allowed"] != "none" else 0)
    if not case["in_place"]:
        n += 2 * N * V * e
    else:
        touched = _distinct(case["L"], V) + case.get("bias", 0)
        n += N * e * (2 * touched + V * (1 - ALLOWED.get(case["allowed"], 1.0)))
    return {"bytes": n, "flops": 6 * N * L + N * V}


# ------------------------------------------------------------------ inputs
def _tokens(g, shape, V):
    """Token ids as texts have them: the r-th most frequent one about 1/r as often as the first."""
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)
    return torch.randperm(V, generator=g, device="cuda")[rank].to(torch.int32)


def _shapes(case):
    """(shape, type) of every gradient, in the order of the layers."""
    d, f, r, t = case["d"], case["f"], case["rank"], case["type"]
    if r:
        return [s for _ in range(4 * case["layers"]) for s in (((r, d), t), ((d, r), t))]
    layer = [((d,), t), ((d, d), t), ((2 * (d // 4), d), t), ((d, d), t), ((d,), t), ((2 * f, d), t), ((d, f), t)]
    return [((case["V"], d), "fp32")] + layer * case["layers"] + [((d,), t)]


def _history(g, case):
    """(history [N, L], lengths [N], prompt [N]): of several rows the first has no history."""
    N, L = case["N"], case["L"]
    history = _tokens(g, (N, L), case["V"])
    lengths = torch.randint((L + 1) // 2, L + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
    if N > 1:
        lengths[0] = 0
    prompt = (lengths * torch.rand(N, generator=g, device="cuda")).to(torch.int32)
    return history, lengths, prompt


def _allowed(g, case):
    """Bits [N, ceil(V/32)] of allowed tokens: of several rows the second has none."""
    if case["allowed"] == "none":
        return None
    N, V = case["N"], case["V"]
    keep = torch.rand(N, -(-V // 32) * 32, generator=g, device="cuda") < ALLOWED[case["allowed"]]
    if N > 1:
        keep[1] = False
    powers = torch.ones(32, dtype=torch.int32, device="cuda") << torch.arange(32, device="cuda", dtype=torch.int32)
    return (keep.view(N, -1, 32) * powers).sum(2, dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] in ("embed", "embed_grad"):
        N, d, V, t = case["N"], case["d"], case["V"], TYPES[case["type"]]
        s["scale"] = math.sqrt(d)
        s["tokens"] = _tokens(g, (N,), V)
        if N > 1:  # a batch of texts of several lengths: some slots are empty
            s["tokens"][torch.rand(N, generator=g, device="cuda") < 0.03] = EMPTY
        if case["op"] == "embed" or case["what"] == "autograd":
            s["W"] = (torch.randn(V, d, generator=g, device="cuda") / math.sqrt(d)).to(t)
        if case["op"] == "embed_grad":
            s["g"] = (torch.randn(N, d, generator=g, device="cuda") * 1e-3).to(t)
            if case["what"] == "add":
                s["dW"] = torch.randn(V, d, generator=g, device="cuda") * 1e-2
            elif case["what"] == "autograd":
                s["W"].requires_grad_()
        return s
    if case["op"] == "clip":
        shapes = _shapes(case)
        s["grads"] = [(torch.randn(shape, generator=g, device="cuda") * 1e-3).to(TYPES[t]) for shape, t in shapes]
        if case["what"] == "clip":  # where they go: one buffer, as an exchange between ranks has it
            sizes = [x.numel() for x in s["grads"]]
            s["flat"] = torch.empty(sum(sizes), dtype=TYPES[case["out"]], device="cuda")
            s["out"] = [x.view(y.shape) for x, y in zip(s["flat"].split(sizes), s["grads"])]
        return s
    N, V, t = case["N"], case["V"], TYPES[case["type"]]
    s["history"], s["lengths"], s["prompt"] = _history(g, case)
    s["allowed"] = _allowed(g, case)
    s["logits"] = (torch.randn(N, V, generator=g, device="cuda") * 2.5).to(t)
    s["r"] = 1 + 0.3 * torch.rand(N, generator=g, device="cuda")
    if case["op"] == "adjust_grad":
        s["g"] = (torch.randn(N, V, generator=g, device="cuda") * 1e-2).to(t)
        return s
    s["f"] = torch.rand(N, generator=g, device="cuda")
    s["p"] = torch.rand(N, generator=g, device="cuda")
    s["bias_tokens"] = s["bias"] = None
    if case["bias"]:
        s["bias_tokens"] = torch.randint(-1, V, (N, case["bias"]), generator=g, device="cuda", dtype=torch.int32)
        s["bias"] = 2 * torch.randn(N, case["bias"], generator=g, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _plain_embed(W, tokens, scale):
    y = W[tokens.clamp(min=0).long()].float() * scale
    return torch.where((tokens == EMPTY)[:, None], torch.zeros_like(y), y).to(W.dtype)


def _plain_embed_grad(tokens, g, V, scale):
    """In 32 bits."""
    live = (tokens != EMPTY)[:, None]
    dW = torch.zeros(V, g.shape[1], device=g.device)
    return dW.index_add_(0, tokens.clamp(min=0).long(), torch.where(live, g.float(), 0.0)) * scale


def _plain_norm(grads):
    return torch.stack([x.float().square().sum() for x in grads]).sum().sqrt().view(1)


def _plain_clip(grads, max_norm, out):
    norm = _plain_norm(grads)
    c = (max_norm / (norm + EPS)).clamp(max=1.0)
    _ = [y.copy_(x.float() * c) for x, y in zip(grads, out)]
    return norm


def _plain_counts(s, V):
    """(seen, how often generated), fp32 [N, V]."""
    h = s["history"]
    at = torch.arange(h.shape[1], device=h.device)
    live = (at < s["lengths"][:, None]) & (h != EMPTY)
    one = torch.ones_like(h, dtype=torch.float32)
    zero = torch.zeros(h.shape[0], V + 1, device=h.device)
    seen = zero.scatter(1, torch.where(live, h, V).long(), one)
    count = zero.scatter_add(1, torch.where(live & (at >= s["prompt"][:, None]), h, V).long(), one)
    return seen[:, :V], count[:, :V]


def _plain_bits(allowed, V):
    v = torch.arange(V, device=allowed.device)
    return (allowed[:, v // 32] >> (v % 32).to(torch.int32)) & 1 == 1


def _plain_adjust(s):
    z = s["logits"].float()
    N, V = z.shape
    seen, count = _plain_counts(s, V)
    r = s["r"][:, None]
    z = torch.where(seen > 0, torch.where(z > 0, z / r, z * r), z)
    z = z - s["f"][:, None] * count - s["p"][:, None] * (count > 0)
    if s["bias"] is not None:
        at = torch.where(s["bias_tokens"] == EMPTY, V, s["bias_tokens"]).long()
        z = z + torch.zeros(N, V + 1, device=z.device).scatter_add_(1, at, s["bias"])[:, :V]
    if s["allowed"] is not None:
        z = torch.where(_plain_bits(s["allowed"], V), z, -math.inf)
    return s["logits"].copy_(z) if s["in_place"] else z.to(s["logits"].dtype)


def _plain_adjust_grad(s):
    z, g = s["logits"].float(), s["g"].float()
    seen, _ = _plain_counts(s, z.shape[1])
    r = s["r"][:, None]
    dz = torch.where(seen > 0, torch.where(z > 0, g / r, g * r), g)
    if s["allowed"] is not None:
        dz = torch.where(_plain_bits(s["allowed"], z.shape[1]), dz, torch.zeros_like(dz))
    return s["g"].copy_(dz) if s["in_place"] else dz.to(s["g"].dtype)


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "embed":
        return _plain_embed(s["W"], s["tokens"], s["scale"])
    if s["op"] == "embed_grad":
        dW = _plain_embed_grad(s["tokens"], s["g"], s["V"], s["scale"])
        if s["what"] == "add":
            return s["dW"].add_(dW)
        if s["what"] == "autograd":
            return _plain_embed(s["W"].detach(), s["tokens"], s["scale"]), dW.to(TYPES[s["out"]])
        return dW.to(TYPES[s["out"]])
    if s["op"] == "clip":
        if s["what"] == "norm":
            return _plain_norm(s["grads"])
        return _plain_clip(s["grads"], s["max_norm"], s["out"]), s["flat"]
    return _plain_adjust(s) if s["op"] == "adjust" else _plain_adjust_grad(s)


def _run_own(s):
    import chunked_kl_loss_gb300 as fckl
    if s["op"] == "embed":
        return fckl.embedding(s["W"], s["tokens"], scale=s["scale"])
    if s["op"] == "embed_grad":
        if s["what"] == "add":
            return fckl.embedding_backward(s["g"], s["tokens"], s["V"], scale=s["scale"], dW=s["dW"], accumulate=True)
        if s["what"] == "autograd":
            y = fckl.differentiable_embedding(s["W"], s["tokens"], scale=s["scale"])
            return y.detach(), torch.autograd.grad(y, s["W"], s["g"])[0]
        return fckl.embedding_backward(s["g"], s["tokens"], s["V"], scale=s["scale"], dtype=TYPES[s["out"]])
    if s["op"] == "clip":
        if s["what"] == "norm":
            return fckl.gradient_norm(s["grads"])
        return fckl.clip_gradients(s["grads"], s["max_norm"], out=s["out"]), s["flat"]
    if s["op"] == "adjust":
        return fckl.adjust_logits(s["logits"], s["history"], s["lengths"], s["prompt"], repetition=s["r"],
                                  frequency=s["f"], presence=s["p"], bias_tokens=s["bias_tokens"], bias=s["bias"],
                                  allowed=s["allowed"], out=s["logits"] if s["in_place"] else None)
    return fckl.adjust_logits_backward(s["g"], s["logits"], s["history"], s["lengths"], repetition=s["r"],
                                       allowed=s["allowed"], out=s["g"] if s["in_place"] else None)


# ------------------------------------------------------------------ 64 bits
def _exact_dW(s):
    """Sums of the gradient rows by token, one column block after the other."""
    V, d = s["V"], s["d"]
    dW = torch.zeros(V + 1, d, dtype=torch.float64, device="cuda")  # the last row takes the empty slots
    at = torch.remainder(s["tokens"].long(), V + 1)
    dW.index_put_((at,), s["g"].double(), accumulate=True)
    return dW[:V].mul_(s["scale"])


def _exact_repeats(s, first):
    """How often each token stands in the history from entry `first` on, by one number per (row, token)."""
    N, V = s["N"], s["V"]
    row = torch.repeat_interleave(torch.arange(N, device="cuda"), (s["lengths"] - first).long())
    at = torch.arange(row.numel(), device="cuda") - torch.cumsum((s["lengths"] - first).long(), 0)[row] + s["lengths"].long()[row]
    key = row * V + s["history"][row, at].long()
    return torch.bincount(key, minlength=N * V).view(N, V)


def _exact_keep(s):
    bits = s["allowed"][:, :, None].bitwise_and(torch.tensor([1 << i if i < 31 else -(1 << 31) for i in range(32)],
                                                             dtype=torch.int32, device="cuda"))
    return bits.ne(0).view(s["N"], -1)[:, :s["V"]]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("embed", "embed_grad"):
        with torch.no_grad():
            y = dW = None
            if "W" in s:
                rows = s["W"].detach().index_select(0, s["tokens"].relu().long()).double()
                y = rows * s["tokens"].ge(0).double().mul(s["scale"])[:, None]
            if case["op"] == "embed":
                return y
            dW = _exact_dW(s)
        if case["what"] == "add":
            return dW.add_(s["dW"].double())
        return dW if y is None else (y, dW)
    if case["op"] == "clip":
        total = sum(float(x.double().norm()) ** 2 for x in s["grads"])
        norm = torch.tensor([math.sqrt(total)], dtype=torch.float64, device="cuda")
        if case["what"] == "norm":
            return norm
        c = min(1.0, case["max_norm"] / (math.sqrt(total) + EPS))
        return norm, torch.cat([x.double().flatten() * c for x in s["grads"]])
    z = s["logits"].double()
    r = s["r"].double()[:, None]
    slope = torch.where(_exact_repeats(s, 0 * s["lengths"]) > 0, torch.where(z > 0, 1 / r, r), 1.0)
    if case["op"] == "adjust_grad":
        dz = slope.mul_(s["g"].double())
        return dz if s["allowed"] is None else dz.masked_fill_(~_exact_keep(s), 0.0)
    z.mul_(slope)
    repeats = _exact_repeats(s, s["prompt"])
    z -= repeats * s["f"].double()[:, None] + repeats.clamp(max=1) * s["p"].double()[:, None]
    if s["bias"] is not None:
        at = s["bias_tokens"].long()
        row = torch.arange(case["N"], device="cuda")[:, None].expand_as(at)
        z.index_put_((row[at >= 0], at[at >= 0]), s["bias"].double()[at >= 0], accumulate=True)
    return z if s["allowed"] is None else z.masked_fill_(~_exact_keep(s), -math.inf)
