"""The serving head's operators as cases that can be timed and compared: the final RMS norm with
the residual's addition (8-bit output, or bf16 with its backward pass), the 8-bit quantisation of
the head's weight, the 8-bit logits product with a scale per block of 128, and sampling from the
logits with given uniform numbers.

``run`` computes an operator in plain torch operations, or, where ``own`` is set, through this
package's entry points. All tensors are on the current CUDA device."""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # a block whose values are all smaller is scaled as if this were its largest
BLOCK = 128


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the final norm of one decoded token, feeding the 8-bit head
        dict(name="norm8 decode", op="norm8", N=1, d=4096),
        # the same after a prompt whose rows are all scored
        dict(name="norm8 prompt", op="norm8", N=4096, d=5120),
        # a training step's norm, forward and backward, at the large-vocabulary step's rows
        dict(name="norm train", op="norm_train", N=8192, d=4096),
        # a short ragged batch with an odd hidden size (21 x 64)
        dict(name="norm train ragged", op="norm_train", N=515, d=1344),
        # loading a checkpoint: a ragged vocabulary and a last block of 64 columns
        dict(name="quantize ragged", op="quantize", rows=50001, d=2112, block_rows=128),
        # the largest head of the workloads
        dict(name="quantize large", op="quantize", rows=151936, d=5120, block_rows=128),
        # logits of one token, small model
        dict(name="logits decode", op="logits", N=1, V=32000, d=2048, out="float32"),
        # a decode batch on a large vocabulary
        dict(name="logits batch", op="logits", N=64, V=128256, d=4096, out="float32"),
        # scoring a prompt with the logits kept in bf16
        dict(name="logits prompt", op="logits", N=4096, V=32000, d=2048, out="bfloat16"),
        # one token with one set of sampling parameters
        dict(name="sample one", op="sample", N=1, V=32000, dtype="float32", mode="scalars", masked=False),
        # a decode batch in which every request brings its own parameters
        dict(name="sample batch", op="sample", N=256, V=151936, dtype="float32", mode="per row", masked=False),
        # bf16 logits of an odd vocabulary, a third of it masked out by a grammar
        dict(name="sample masked", op="sample", N=33, V=50001, dtype="bfloat16", mode="per row", masked=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm8", "norm_train", "quantize", "logits", "logits", "sample", "sample"])
    d = 64 * _log_int(rng, 4, 80)
    if op in ("norm8", "norm_train"):
        return dict(op=op, N=_log_int(rng, 1, min(8192, 8192 * 4096 // d)), d=d)
    if op == "quantize":
        return dict(op=op, rows=_log_int(rng, 1, 151936), d=d, block_rows=rng.choice([1, 128]))
    if op == "logits":
        V = _log_int(rng, 1000, 151936)
        most = min(4096, max(1, (4096 * 32000 * 2048) // (V * d)))
        return dict(op=op, N=_log_int(rng, 1, most), V=V, d=d, out=rng.choice(["float32", "bfloat16"]))
    return dict(op=op, N=_log_int(rng, 1, 256), V=_log_int(rng, 500, 151936), dtype=rng.choice(["float32", "bfloat16"]),
                mode=rng.choice(["plain", "scalars", "per row"]), masked=rng.random() < 0.3)


# ------------------------------------------------------------------------------------ inputs

def _blocks(n):
    return -(-n // BLOCK)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, bf = case["op"], torch.bfloat16

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(bf)

    s = dict(case=case)
    if op in ("norm8", "norm_train"):
        N, d = case["N"], case["d"]
        # a residual stream a few times larger than what the last layer adds, some channels far larger
        channel = torch.exp(0.7 * torch.randn(d, device="cuda", generator=g))
        s["residual"] = (torch.randn(N, d, device="cuda", generator=g) * 3 * channel).to(bf)
        s["x"] = normal(N, d)
        s["weight"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(bf)
        s["eps"] = 1e-6
        if op == "norm_train":
            s["dy"] = normal(N, d, scale=1e-3)
            s["dsum"] = normal(N, d, scale=1e-3)
    elif op == "quantize":
        s["W"] = torch.randn(case["rows"], case["d"], device="cuda", generator=g, dtype=bf) * 0.02
    elif op == "logits":
        N, V, d = case["N"], case["V"], case["d"]
        s["H8"], s["h_scale"] = _quantize(torch.randn(N, d, device="cuda", generator=g, dtype=bf), 1)
        W = torch.randn(V, d, device="cuda", generator=g, dtype=bf) * 0.02
        s["W8"], s["w_scale"] = _quantize(W, BLOCK)
    else:
        N, V = case["N"], case["V"]
        # rows between flat and sharply peaked, frequent tokens likelier than rare ones
        z = torch.randn(N, V, device="cuda", generator=g)
        z *= 1 + 2.5 * torch.rand(N, 1, device="cuda", generator=g)
        z -= 0.6 * torch.log1p(torch.randperm(V, device="cuda", generator=g).float())
        if case["masked"]:
            z.masked_fill_(torch.rand(N, V, device="cuda", generator=g) < 0.33, -math.inf)
            z[:, 0] = 0.0  # a mask leaves something
        s["logits"] = z.to(getattr(torch, case["dtype"]))
        s["u"] = torch.rand(N, device="cuda", generator=g)
        s["params"] = dict(temperature=None, top_k=None, top_p=None, min_p=None)
        if case["mode"] == "scalars":
            s["params"] = dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)
        elif case["mode"] == "per row":
            def pick(values, dtype):
                i = torch.randint(len(values), (N,), device="cuda", generator=g)
                return torch.tensor(values, device="cuda", dtype=dtype)[i]
            f = torch.float32
            s["params"] = dict(temperature=pick([0.5, 0.7, 1.0, 1.3], f), top_k=pick([0, 0, 1, 20, 50, 1000], torch.int32),
                               top_p=pick([1.0, 1.0, 0.5, 0.9, 0.95], f), min_p=pick([0.0, 0.0, 0.02, 0.1], f))
    return s


# ------------------------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import lm_head_cross_tcgen05_b200 as lmh

    op = s["case"]["op"]
    if op == "norm8":
        o = lmh.rms_norm(s["x"], s["weight"], s["residual"], eps=s["eps"], fp8=True)
        return dict(sum=o["sum"], q=o["q"], scale=o["scale"])
    if op == "norm_train":
        f = lmh.rms_norm(s["x"], s["weight"], s["residual"], eps=s["eps"])
        b = lmh.rms_norm_bwd(f["sum"], s["weight"], f["rstd"], s["dy"], s["dsum"])
        return dict(sum=f["sum"], y=f["y"], dx=b["dx"], dweight=b["dweight"])
    if op == "quantize":
        q, scale = lmh.quantize_fp8(s["W"], s["case"]["block_rows"])
        return dict(q=q, scale=scale)
    if op == "logits":
        o = lmh.fp8_logits(s["H8"], s["h_scale"], s["W8"], s["w_scale"], dtype=getattr(torch, s["case"]["out"]))
        return dict(logits=o["logits"])
    o = lmh.sample(s["logits"], s["u"], **s["params"])
    return dict(tokens=o["tokens"], logprob=o["logprob"])


def _quantize(x, block_rows):
    """e4m3 values and one scale per block of block_rows x 128."""
    rows, d = x.shape
    R, C = -(-rows // block_rows), _blocks(d)
    a = torch.nn.functional.pad(x.float(), (0, C * BLOCK - d, 0, R * block_rows - rows))
    a = a.view(R, block_rows, C, BLOCK)
    scale = a.abs().amax(dim=(1, 3)).clamp(min=AMAX_FLOOR) / E4M3_MAX
    q = (a / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(R * block_rows, C * BLOCK)[:rows, :d].contiguous(), scale


def _expand(scale, block_rows, rows, d):
    return scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :d]


def _params(s):
    """Every row's parameters, as the 32-bit values that the entries take: those that are off are one or zero."""
    n, p = s["logits"].shape[0], s["params"]

    def rows(v, default, dtype):
        v = default if v is None else v
        return v if isinstance(v, torch.Tensor) else torch.full((n,), v, device="cuda", dtype=dtype)
    f = torch.float32
    return (rows(p["temperature"], 1.0, f).double(), rows(p["top_k"], 0, torch.int32).long(), rows(p["top_p"], 1.0, f).double(),
            rows(p["min_p"], 0.0, f).double())


def _plain(s):
    op = s["case"]["op"]
    if op in ("norm8", "norm_train"):
        total = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)  # the stream as it is stored
        t, w = total.float(), s["weight"].float()
        rstd = torch.rsqrt(t.square().mean(1, keepdim=True) + s["eps"])
        n = t * rstd
        y = n * w
        if op == "norm8":
            q, scale = _quantize(y, 1)
            return dict(sum=total, q=q, scale=scale)
        dy = s["dy"].float()
        wdy = dy * w
        dx = (wdy - n * (wdy * n).mean(1, keepdim=True)) * rstd + s["dsum"].float()
        dweight = (dy * n).sum(0)
        return dict(sum=total, y=y.to(torch.bfloat16), dx=dx.to(torch.bfloat16), dweight=dweight.to(torch.bfloat16))
    if op == "quantize":
        q, scale = _quantize(s["W"], s["case"]["block_rows"])
        return dict(q=q, scale=scale)
    if op == "logits":
        (N, d), V = s["H8"].shape, s["W8"].shape[0]
        h = s["H8"].float() * _expand(s["h_scale"], 1, N, d)
        w = s["W8"].float() * _expand(s["w_scale"], BLOCK, V, d)
        return dict(logits=(h @ w.t()).to(getattr(torch, s["case"]["out"])))
    # sampling, in 64 bits: a token changes where a sum of probabilities crosses a border
    z, (tau, k, p, m) = s["logits"].double(), _params(s)
    V = z.shape[1]
    top = z.amax(1, keepdim=True)
    t = (z - top) / tau[:, None]
    e = t.exp()
    order = torch.sort(z, dim=1, descending=True, stable=True).indices  # equal logits: the lowest index first
    rank = torch.arange(V, device=z.device)[None]
    k = torch.where((k <= 0) | (k > V), V, k)[:, None]
    es = torch.where(rank < k, e.gather(1, order), 0.0)
    cum = es.cumsum(1)
    before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1)
    p = p[:, None]
    keep = (rank < k) & ((p >= 1) | (rank == 0) | (before < p * cum[:, -1:]))
    keep = torch.zeros_like(keep).scatter_(1, order, keep)
    keep &= t >= m[:, None].log()
    c = torch.where(keep, e, 0.0).cumsum(1)
    token = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(1)
    logprob = t.gather(1, token[:, None])[:, 0] - e.sum(1).log()
    return dict(tokens=token.int(), logprob=logprob.float())


# ------------------------------------------------------------------------------------ what a pass needs

def work(case):
    op = case["op"]
    if op in ("norm8", "norm_train"):
        N, d = case["N"], case["d"]
        if op == "norm8":  # x, residual; sum, 8-bit values and scales
            return dict(bytes=N * d * 7 + N * _blocks(d) * 4 + d * 2, flops=N * d * 7)
        # in: x, residual, dy, dsum, weight; out: sum, y, dx and the weight's gradient
        return dict(bytes=N * d * 14 + d * 4, flops=N * d * 16)
    if op == "quantize":
        n, d = case["rows"], case["d"]
        return dict(bytes=n * d * 3 + -(-n // case["block_rows"]) * _blocks(d) * 4, flops=n * d * 2)
    if op == "logits":
        N, V, d = case["N"], case["V"], case["d"]
        out = 4 if case["out"] == "float32" else 2
        return dict(bytes=(N + V) * d + (N + _blocks(V)) * _blocks(d) * 4 + N * V * out, flops=2 * N * V * d)
    N, V = case["N"], case["V"]
    return dict(bytes=N * V * (4 if case["dtype"] == "float32" else 2) + N * 28, flops=N * V * 8)


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definitions in 64 bits. 8-bit values are given before their rounding."""
    s = prepare(case, seed)
    op = case["op"]

    def by_block(a, rows):
        n, d = a.shape
        scale = torch.empty(-(-n // rows), _blocks(d), dtype=torch.float64, device="cuda")
        q = torch.empty_like(a)
        for j in range(_blocks(d)):
            part = a[:, j * BLOCK:(j + 1) * BLOCK]
            high = part.abs().max(dim=1).values
            high = torch.cat([high, high.new_zeros(scale.shape[0] * rows - n)]).view(-1, rows).max(dim=1).values
            scale[:, j] = torch.maximum(high, torch.tensor(AMAX_FLOOR, dtype=torch.float64, device="cuda")) / E4M3_MAX
            q[:, j * BLOCK:(j + 1) * BLOCK] = part / scale[:, j].repeat_interleave(rows)[:n, None]
        return q, scale

    if op in ("norm8", "norm_train"):
        a = s["x"].double() + s["residual"].double()
        r = a.to(torch.bfloat16).double()  # the norm is that of the stored sum
        w, d = s["weight"].double(), case["d"]
        ms = torch.linalg.vector_norm(r, dim=1) ** 2 / d + s["eps"]
        y = w * r / ms.sqrt()[:, None]
        if op == "norm8":
            q, scale = by_block(y, 1)
            return dict(sum=a, q=q, scale=scale)
        gy = s["dy"].double()
        # y_j = w_j r_j ms^(-1/2);  dms/dr_i = 2 r_i / d
        dot = torch.einsum("nd,nd,d->n", gy, r, w)
        dx = gy * w / ms.sqrt()[:, None] - r * (dot / (d * ms ** 1.5))[:, None] + s["dsum"].double()
        return dict(sum=a, y=y, dx=dx, dweight=torch.einsum("nd,nd,n->d", gy, r, ms ** -0.5))
    if op == "quantize":
        q, scale = by_block(s["W"].double(), case["block_rows"])
        return dict(q=q, scale=scale)
    if op == "logits":
        N, V, d = case["N"], case["V"], case["d"]
        z = torch.zeros(N, V, dtype=torch.float64, device="cuda")
        for j in range(_blocks(d)):
            c = slice(j * BLOCK, (j + 1) * BLOCK)
            part = s["H8"][:, c].double() @ s["W8"][:, c].double().t()
            z += part * s["h_scale"][:, j].double()[:, None] * s["w_scale"][:, j].double().repeat_interleave(BLOCK)[:V]
        return dict(logits=z)
    tau, ks, ps, ms = (v.tolist() for v in _params(s))
    tokens, logprob = [], []
    for i, u in enumerate(s["u"].tolist()):
        z = s["logits"][i].double() / tau[i]
        v, idx = torch.sort(-z, stable=True)
        e = torch.exp(v[0] - v)
        n = ks[i] if 0 < ks[i] < z.numel() else z.numel()
        c = torch.cumsum(e[:n], 0)
        if ps[i] < 1:
            n = min(n, int(torch.searchsorted(c, ps[i] * c[-1])) + 1)
        if ms[i] > 0:
            n = min(n, int((v - v[0] <= -math.log(ms[i])).sum()))
        ids = torch.sort(idx[:n]).values
        c = torch.cumsum(torch.exp(z[ids] + v[0]), 0)
        t = int(ids[min(n - 1, int(torch.searchsorted(c, u * c[-1], right=True)))])
        tokens.append(t)
        logprob.append(float(z[t] - torch.logsumexp(z, 0)))
    return dict(tokens=torch.tensor(tokens, dtype=torch.int32), logprob=torch.tensor(logprob, dtype=torch.float64))
