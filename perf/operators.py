"""The operators that fine-tune and serve an MoE layer around its frozen experts, as cases to measure.

Five operators, each in its plain form (elementary torch operations in 32 bits, rounded once) and as
the library's call:

  balance           the router's balance loss over sequences, with per-expert counts
  router_backward   gradient of the router's logits: gates and balance loss in one pass
  lora              low-rank adapters of many requests beside one projection: out = base + s (x A^T) B^T
  lora_backward     the adapters' gradients and the input's
  combine_backward  gradients of the expert outputs and of the gate weights

Sizes are those of the library's layers (4096 tokens of 4096 or 7168 columns, 8 / 64 / 128 / 256 experts,
decode batches of 128 tokens with 2048 columns) and ragged ones around them.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
ALPHA = 0.01  # weight of the balance loss


# ---------------------------------------------------------------- cases
def _router(name, op, T, E, k, S, dtype, mask=False, renorm=False, out="f32"):
    return dict(name=name, op=op, T=T, E=E, k=k, S=S, dtype=dtype, mask=mask, renorm=renorm, out=out)


def _lora(name, op, T, Q, n, R, d, N, out, bare=False):
    return dict(name=name, op=op, T=T, Q=Q, n=n, R=R, d=d, N=N, out=out, bare=bare)


def _combine(name, T, d, k, shared, dtype):
    return dict(name=name, op="combine_backward", T=T, d=d, k=k, shared=shared, dtype=dtype)


def listed():
    return [
        # one decode step's batch, 64 experts top-2: the launch is what counts
        _router("balance decode", "balance", 128, 64, 2, 1, "f32"),
        # a long training batch of ragged sequences with padded tokens, 128 experts top-4, 16-bit logits
        _router("balance sequences", "balance", 65536, 128, 4, 37, "f16", mask=True),
        # the fine-grained layer's router: 256 experts top-8, a handful of sequences
        _router("router gradient fine", "router_backward", 4096, 256, 8, 5, "f32"),
        # the long batch, renormalised gates, 16-bit logits and gradient
        _router("router gradient long", "router_backward", 65536, 128, 4, 1, "bf16", mask=True, renorm=True, out="bf16"),
        # decode: one token per request, nearly every one with an adapter of its own, gate-and-up width
        _lora("adapters decode", "lora", 61, 61, 48, 16, 2048, 2816, "bf16", bare=True),
        # a mixed step: a few prompts of odd lengths, some without an adapter, high rank
        _lora("adapters mixed", "lora", 1021, 19, 12, 64, 4096, 4096, "bf16", bare=True),
        # prefill of long prompts beside the wide hidden size
        _lora("adapters prefill", "lora", 8192, 24, 8, 32, 7168, 4096, "bf16"),
        # a small training step of three adapters on narrow odd widths, 32-bit activations' gradient
        _lora("adapter gradients small", "lora_backward", 203, 5, 3, 8, 1408, 2048, "f32", bare=True),
        # one adapter trained on a whole batch
        _lora("adapter gradients one", "lora_backward", 4096, 4, 1, 16, 4096, 4096, "bf16"),
        # many users' adapters trained together, high rank, down projection
        _lora("adapter gradients many", "lora_backward", 8191, 40, 16, 64, 2048, 7168, "bf16"),
        # a decode-shaped layer
        _combine("combine gradient decode", 128, 2048, 2, False, "bf16"),
        # the fine-grained layer with its shared expert
        _combine("combine gradient fine", 4096, 7168, 8, True, "bf16"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["balance", "router_backward", "lora", "lora_backward", "combine_backward"])
    if op in ("balance", "router_backward"):
        T, E = _log(rng, 1, 65536), _log(rng, 4, 512)
        T = min(T, 65536 * 128 // E)
        c = _router("", op, T, E, rng.randint(1, min(8, E)), _log(rng, 1, 64), rng.choice(["f32", "f16", "bf16"]),
                    rng.random() < 0.5, rng.random() < 0.5, rng.choice(["f32", "bf16"]))
    elif op == "combine_backward":
        T, d, k = _log(rng, 1, 8192), _log(rng, 64, 7168, 8), rng.randint(1, 8)
        T = min(T, 4096 * 7168 * 9 // (d * (k + 1)))
        c = _combine("", T, d, k, rng.random() < 0.5, rng.choice(["f32", "bf16"]))
    else:
        T, R = _log(rng, 1, 8192), rng.choice([8, 16, 24, 32, 64])
        d, N = _log(rng, 64, 7168, 8), _log(rng, 64, 7168, 8)
        n = _log(rng, 1, 128)
        n = max(1, min(n, int(2.0e10 / (T * R * (d + N)))))
        c = _lora("", op, T, _log(rng, 1, min(T, 256)), n, R, d, N, rng.choice(["f32", "bf16"]), rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _cuts(rng, T, parts):
    """Ragged lengths of `parts` runs that cover T."""
    marks = sorted(rng.randint(0, T) for _ in range(parts - 1))
    return [b - a for a, b in zip([0] + marks, marks + [T])]


def _offsets(lengths):
    o = [0]
    for n in lengths:
        o.append(o[-1] + n)
    return o


def _router_state(case, seed, g, rng):
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    used = T - T // 50 if case["mask"] else T  # rows behind the last sequence are padding
    offsets = _offsets(_cuts(rng, used, S))
    # popular experts, as an untuned router has them
    lean = -0.7 * torch.log1p(torch.randperm(E, generator=g, device="cuda").float())
    logits = (torch.randn(T, E, generator=g, device="cuda") + lean).to(DTYPES[case["dtype"]])
    s = dict(case=case, logits=logits, idx=torch.topk(logits.float(), k, dim=1).indices.to(torch.int32).contiguous(),
             offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), mask=None)
    if case["mask"]:
        s["mask"] = (torch.rand(T, generator=g, device="cuda") > 0.05).to(torch.uint8)
    if case["op"] == "router_backward":
        s["d_w"] = torch.randn(T, k, generator=g, device="cuda") * 0.1
        s["d_loss"] = torch.full((1,), 1.0, device="cuda")
        # what the loss's forward left: counts and each sequence's coefficient
        counts, tokens = _counts(s)
        live = (tokens > 0).sum().clamp(min=1)
        s["counts"] = counts
        s["coef"] = torch.where(tokens > 0, ALPHA * E / (k * tokens.double().clamp(min=1) ** 2 * live), 0.0).float()
    return s


def _lora_state(case, seed, g, rng):
    T, Q, n, R, d, N = (case[v] for v in ("T", "Q", "n", "R", "d", "N"))
    lengths = [v + 1 for v in _cuts(rng, T - Q, Q)]
    ids = list(range(n))
    rng.shuffle(ids)
    at = [-1 if case["bare"] and q % 8 == 7 else ids[q % n] for q in range(Q)]
    row = torch.repeat_interleave(torch.tensor(at, dtype=torch.int32), torch.tensor(lengths)).cuda()
    # the plan a batch's every projection shares: rows in adapter order, those without one last
    key = torch.where(row < 0, n, row).long()
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    ends = torch.cumsum(torch.bincount(key, minlength=n + 1)[:n], 0)
    s = dict(case=case, row=row, order=order, offsets=torch.cat([ends.new_zeros(1), ends]).to(torch.int32))

    def normal(*shape, std=1.0):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)

    s["x"] = normal(T, d)
    s["A"], s["B"] = normal(n, R, d, std=1 / math.sqrt(d)), normal(n, N, R, std=0.1)
    s["scale"] = torch.rand(n, generator=g, device="cuda") + 0.5
    t = DTYPES[case["out"]]
    if case["op"] == "lora":
        s["base"] = normal(T, N).to(t)
        s["out"] = torch.empty(T, N, dtype=t, device="cuda")
    else:
        s["dC"] = normal(T, N, std=0.1)
        s["dx_base"] = normal(T, d, std=0.1).to(t)
        a = torch.cat([s["A"], torch.zeros_like(s["A"][:1])])
        h = torch.zeros(T, R, device="cuda")  # the forward's x A^T
        for v in range(n):
            rows = (row == v).nonzero().flatten()
            h[rows] = s["x"][rows].float() @ a[v].float().t()
        s["h"] = h
    return s


def _combine_state(case, seed, g, rng):
    T, d, k = case["T"], case["d"], case["k"]
    rows = T * k + (T if case["shared"] else 0)
    perm = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)  # the permute's plan
    w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), dim=1)
    y = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    d_out = torch.empty(T, d, device="cuda", dtype=DTYPES[case["dtype"]]).normal_(0, 0.1, generator=g)
    return dict(case=case, d_out=d_out, Y=y, t2r=perm.contiguous(), w=w)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    if case["op"] in ("balance", "router_backward"):
        return _router_state(case, seed, g, rng)
    if case["op"] == "combine_backward":
        return _combine_state(case, seed, g, rng)
    return _lora_state(case, seed, g, rng)


# ---------------------------------------------------------------- plain forms
def _live(s):
    """[T] which sequence each token counts for, S where none."""
    T, S = s["case"]["T"], s["case"]["S"]
    t = torch.arange(T, device="cuda")
    seq = torch.bucketize(t, s["offsets"][1:].long(), right=True)
    seq = torch.where(t >= s["offsets"][-1], S, seq)
    return seq if s["mask"] is None else torch.where(s["mask"] != 0, seq, S)


def _counts(s):
    c = s["case"]
    seq = _live(s)
    flat = (seq[:, None] * c["E"] + s["idx"].long()).flatten()
    counts = torch.bincount(flat, minlength=(c["S"] + 1) * c["E"])[: c["S"] * c["E"]]
    return counts.view(c["S"], c["E"]).to(torch.int32), torch.bincount(seq, minlength=c["S"] + 1)[: c["S"]]


def _softmax(logits):
    l = logits.float()
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_balance(s):
    c = s["case"]
    counts, tokens = _counts(s)
    member = (_live(s)[None, :] == torch.arange(c["S"], device="cuda")[:, None]).float()
    sums = member @ _softmax(s["logits"])
    n = tokens.float().clamp(min=1)
    live = (tokens > 0).sum().clamp(min=1)
    coef = torch.where(tokens > 0, ALPHA * c["E"] / (c["k"] * n * n * live), 0.0)
    loss = (coef * (counts.float() * sums).sum(1)).sum().reshape(1)
    return loss, counts, sums / n[:, None], coef


def _plain_router_backward(s):
    c = s["case"]
    p, idx = _softmax(s["logits"]), s["idx"].long()
    w = torch.gather(p, 1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
        slot = w * (s["d_w"] - (w * s["d_w"]).sum(1, keepdim=True))
        g = torch.zeros_like(p).scatter_(1, idx, slot)
    else:
        g = torch.zeros_like(p).scatter_(1, idx, s["d_w"])
        g = p * (g - (w * s["d_w"]).sum(1, keepdim=True))
    seq = _live(s)
    zero = s["coef"].new_zeros(1)
    k = torch.cat([s["coef"] * s["d_loss"], zero])[seq]
    n = torch.cat([s["counts"].float(), s["counts"].new_zeros(1, c["E"]).float()])[seq]
    g = g + k[:, None] * p * (n - (n * p).sum(1, keepdim=True))
    return g.to(DTYPES[c["out"]])


def _own_columns(s, v):
    """v [T, n R] with the columns of other rows' adapters zeroed."""
    c = s["case"]
    mine = s["row"][:, None] == torch.arange(c["n"], device="cuda", dtype=torch.int32)
    return (v.view(c["T"], c["n"], c["R"]) * mine[:, :, None]).view(c["T"], -1)


def _plain_lora(s):
    c = s["case"]
    a = s["A"].float().view(-1, c["d"])
    b = (s["B"].float() * s["scale"][:, None, None]).transpose(1, 2).reshape(-1, c["N"])
    h = _own_columns(s, s["x"].float() @ a.t())
    out = (s["base"].float() + h @ b).to(s["base"].dtype)
    return out, h.view(c["T"], c["n"], c["R"]).sum(1)


def _plain_lora_backward(s):
    c = s["case"]
    n, R = c["n"], c["R"]
    a = s["A"].float().view(-1, c["d"])
    b = (s["B"].float() * s["scale"][:, None, None]).transpose(1, 2).reshape(-1, c["N"])
    dc, x = s["dC"].float(), s["x"].float()
    dh = _own_columns(s, dc @ b.t())
    h = _own_columns(s, (s["h"][:, None, :] * s["scale"][:, None]).reshape(c["T"], -1))
    dx = (s["dx_base"].float() + dh @ a).to(s["dx_base"].dtype)
    da = (dh.t() @ x).view(n, R, c["d"])
    db = (dc.t() @ h).view(c["N"], n, R).transpose(0, 1).contiguous()
    return dx, da, db


def _plain_combine_backward(s):
    c = s["case"]
    g = s["d_out"].float()
    at = s["t2r"].long().flatten()
    dy = torch.empty(s["Y"].shape, dtype=torch.float32, device="cuda")
    dy[at] = (s["w"][:, :, None] * g[:, None, :]).view(-1, c["d"])
    if c["shared"]:
        dy[c["T"] * c["k"]:] = g
    dw = (s["Y"][at].float().view(c["T"], c["k"], c["d"]) * g[:, None, :]).sum(2)
    return dy.to(torch.bfloat16), dw


PLAIN = dict(balance=_plain_balance, router_backward=_plain_router_backward, lora=_plain_lora,
             lora_backward=_plain_lora_backward, combine_backward=_plain_combine_backward)


# ---------------------------------------------------------------- the library's calls
def _library(s):
    import grouped_gemm_03_b200 as gg
    c = s["case"]
    if c["op"] == "balance":
        return gg.balance_loss(s["logits"], s["idx"], ALPHA, seq_offsets=s["offsets"], mask=s["mask"])
    if c["op"] == "router_backward":
        return gg.router_backward(s["logits"], s["idx"], s["d_w"], renormalize=c["renorm"], counts=s["counts"],
                                  coef=s["coef"], d_loss=s["d_loss"], seq_offsets=s["offsets"], mask=s["mask"],
                                  out_dtype=DTYPES[c["out"]])
    if c["op"] == "lora":
        return gg.lora(s["x"], s["A"], s["B"], s["offsets"], s["order"], scale=s["scale"], base=s["base"],
                       out=s["out"], want_h=True)
    if c["op"] == "lora_backward":
        return gg.lora_backward(s["dC"], s["x"], s["h"], s["A"], s["B"], s["offsets"], s["order"], scale=s["scale"],
                                dx_base=s["dx_base"])
    return gg.combine_backward(s["d_out"], s["Y"], s["t2r"], s["w"], c["shared"])


def run(state):
    return _library(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- the work none can do without
def work(case):
    c = case
    if c["op"] in ("balance", "router_backward"):
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        read = T * E * BYTES[c["dtype"]] + T * k * 4 + (T if c["mask"] else 0) + (S + 1) * 4
        if c["op"] == "balance":
            return dict(bytes=read + S * E * 8 + S * 4 + 4, flops=T * E * 5)
        return dict(bytes=read + T * k * 4 + T * E * BYTES[c["out"]] + S * E * 4 + S * 4 + 4, flops=T * E * 10)
    if c["op"] == "combine_backward":
        T, d, k = c["T"], c["d"], c["k"]
        written = T * k + (T if c["shared"] else 0)
        return dict(bytes=T * d * BYTES[c["dtype"]] + T * k * d * 2 + written * d * 2 + T * k * 12, flops=T * k * d * 3)
    T, Q, n, R, d, N, b = c["T"], c["Q"], c["n"], c["R"], c["d"], c["N"], BYTES[c["out"]]
    active = len({q % n for q in range(Q) if not (c["bare"] and q % 8 == 7)})
    weights = active * R * (d + N) * 2
    if c["op"] == "lora":
        return dict(bytes=T * d * 2 + 2 * T * N * b + weights + T * R * 4 + T * 4, flops=2 * T * R * (d + N))
    return dict(bytes=T * N * 2 + T * d * 2 + 2 * T * d * b + weights + T * R * 4 + T * 4 + n * R * (d + N) * 4,
                flops=4 * T * R * (d + N))


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] in ("balance", "router_backward"):
        return _exact_router(c, s)
    if c["op"] == "combine_backward":
        g, w, t2r = s["d_out"].double(), s["w"].double(), s["t2r"].long()
        dy = torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            dy[t2r[:, j]] = w[:, j, None] * g
            dw[:, j] = torch.linalg.vecdot(s["Y"][t2r[:, j]].double(), g)
        if c["shared"]:
            dy[c["T"] * c["k"]:] = g
        return dy, dw
    n, row = c["n"], s["row"]
    if c["op"] == "lora":
        out, h = s["base"].double(), torch.zeros(c["T"], c["R"], dtype=torch.float64, device="cuda")
        for a in range(n):
            r = (row == a).nonzero().flatten()
            h[r] = torch.einsum("td,rd->tr", s["x"][r].double(), s["A"][a].double())
            out[r] += s["scale"][a].double() * torch.einsum("tr,nr->tn", h[r], s["B"][a].double())
        return out, h
    dx = s["dx_base"].double()
    da, db = (torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in ("A", "B"))
    for a in range(n):
        r = (row == a).nonzero().flatten()
        dc, sc = s["dC"][r].double(), s["scale"][a].double()
        dh = sc * torch.einsum("tn,nr->tr", dc, s["B"][a].double())
        dx[r] += torch.einsum("tr,rd->td", dh, s["A"][a].double())
        da[a] = torch.einsum("tr,td->rd", dh, s["x"][r].double())
        db[a] = sc * torch.einsum("tn,tr->nr", dc, s["h"][r].double())
    return dx, da, db


def _exact_router(c, s):
    E, k, S = c["E"], c["k"], c["S"]
    l = s["logits"].double()
    p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    bounds = s["offsets"].tolist()
    keep = torch.ones(c["T"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"].bool()
    idx = s["idx"].long()
    hot = torch.zeros(c["T"], E, dtype=torch.float64, device="cuda")
    if c["op"] == "balance":
        hot.scatter_(1, idx, 1.0)
        counts = torch.zeros(S, E, dtype=torch.float64, device="cuda")
        mean, tokens = torch.zeros_like(counts), []
        for q in range(S):
            m = keep[bounds[q]:bounds[q + 1]]
            tokens.append(int(m.sum()))
            if tokens[-1]:
                counts[q] = hot[bounds[q]:bounds[q + 1]][m].sum(0)
                mean[q] = p[bounds[q]:bounds[q + 1]][m].mean(0)
        live = max(1, sum(n > 0 for n in tokens))
        coef = torch.tensor([ALPHA * E / (k * n * n * live) if n else 0.0 for n in tokens], dtype=torch.float64, device="cuda")
        loss = sum(ALPHA * E / live * float((counts[q] / (k * n) * mean[q]).sum()) for q, n in enumerate(tokens) if n)
        return torch.tensor([loss], dtype=torch.float64, device="cuda"), counts.to(torch.int32), mean, coef
    d_w = s["d_w"].double()
    w = torch.gather(p, 1, idx)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        d_p = hot.scatter_(1, idx, d_w / total - (d_w * w).sum(1, keepdim=True) / total ** 2)
    else:
        d_p = hot.scatter_(1, idx, d_w)
    for q in range(S):
        m = keep[bounds[q]:bounds[q + 1]].double()[:, None]
        d_p[bounds[q]:bounds[q + 1]] += m * s["coef"][q].double() * s["d_loss"].double() * s["counts"][q].double()
    return p * (d_p - (p * d_p).sum(1, keepdim=True))
