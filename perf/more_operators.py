"""The operators that train and score a model around the packed layers, as measured cases.

Two operators and their gradients, each with a plain form in elementary torch operations
(fp32, rounded once at the end) and the library's call:

- ``loss`` / ``loss_grad``: softmax cross entropy over a packed output head, z = x W^T,
  loss = log sum_v exp(z_v) - z_target, without the logits, and its gradients with respect
  to the input and to the groups' scales and biases of the head;
- ``norm`` / ``norm_grad``: what stands between two blocks of a model, in one pass over a
  row: the norm after a block, its gate, the residual sum with its factor and the norm
  before the next block,
      t = y / rms(y) * (post + offset),  s = x + factor * gate * t,
      a = s / rms(s) * (weight + offset),  rms(v) = sqrt(mean(v^2) + eps),
  and the gradients of x, y, the two weights and the gate.

W[n, k] = q[n, k] * scale[n, k // group] + bias[n, k // group], code k of a row at bit
k * bits of the row's little-endian 32-bit words.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def _loss(name, op, m, k, v, bits, group, dtype):
    return {"name": name, "op": op, "m": m, "k": k, "v": v, "bits": bits, "group": group, "dtype": dtype}


def _norm(name, op, m, d, dtype, stream, post, gates, pre, offset):
    """gates: rows of the gate (0: none, 1: one for all rows, m: one each, or a divisor of m)."""
    return {"name": name, "op": op, "m": m, "d": d, "dtype": dtype, "stream": stream, "post": post, "gates": gates,
            "pre": pre, "offset": offset}


def listed():
    return [
        # The log-probability of one token that a decoding sequence has taken.
        _loss("loss_1", "loss", 1, 4096, 32000, 4, 64, "bf16"),
        # Scoring one step of a batch of sequences over a large vocabulary, 8 bits.
        _loss("loss_12", "loss", 12, 2048, 131071, 8, 32, "f16"),
        # The loss of a small fp32 model over an uneven batch.
        _loss("loss_200_f32", "loss", 200, 768, 32000, 3, 32, "f32"),
        # The loss of a training step.
        _loss("loss_4096", "loss", 4096, 4096, 32000, 4, 64, "bf16"),
        # A short odd sequence's gradient on a small model, 6-bit codes across words.
        _loss("loss_grad_77", "loss_grad", 77, 1024, 50001, 6, 32, "f16"),
        # The gradient of a training step over a large vocabulary.
        _loss("loss_grad_2048", "loss_grad", 2048, 4096, 131072, 4, 64, "bf16"),
        # One decoded token: both norms, the residual sum.
        _norm("norm_1", "norm", 1, 4096, "bf16", "bf16", True, 0, True, 0.0),
        # A training step's rows, both norms and a gate for each channel.
        _norm("norm_8192", "norm", 8192, 4096, "bf16", "bf16", True, 1, True, 0.0),
        # Four sequences with a gate of their own each, the stream kept in fp32, an odd width.
        _norm("norm_1000_f32", "norm", 1000, 2881, "f16", "f32", True, 4, True, 1.0),
        # A plain residual sum with its norm, the stream in fp32, backward.
        _norm("norm_grad_77", "norm_grad", 77, 5120, "bf16", "f32", False, 0, True, 0.0),
        # A training step's backward pass through both norms, the gate and the sum.
        _norm("norm_grad_8192", "norm_grad", 8192, 4096, "bf16", "bf16", True, 1, True, 0.0),
        # Backward with a gate for each token.
        _norm("norm_grad_600", "norm_grad", 600, 1027, "f16", "f16", True, 600, True, 1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["loss", "loss_grad", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("loss", "loss_grad"):
        group = rng.choice([32, 64, 128])
        return {"op": op, "m": _log_int(rng, 1, 2048), "k": max(1, _log_int(rng, 128, 4096) // group) * group,
                "v": _log_int(rng, 1000, 131072), "bits": rng.choice([2, 3, 4, 4, 6, 8]), "group": group,
                "dtype": dtype}
    m = _log_int(rng, 1, 8192)
    gates = rng.choice([0, 1, m, 4])
    if gates == 4:
        m = 4 * max(1, m // 4)
    post = rng.choice([False, True])
    return {"op": op, "m": m, "d": _log_int(rng, 64, 8192), "dtype": dtype, "stream": rng.choice([dtype, "f32"]),
            "post": post, "gates": gates, "pre": rng.choice([True, True, False]), "offset": rng.choice([0.0, 1.0])}


# ------------------------------------------------------------------ inputs

class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def normal(self, shape, sigma, dtype=torch.float32):
        return (torch.randn(shape, generator=self.g, device=DEV) * sigma).to(dtype)

    def uniform(self, shape, lo, hi):
        return torch.rand(shape, generator=self.g, device=DEV) * (hi - lo) + lo

    def ints(self, shape, lo, hi, dtype=torch.int32):
        return torch.randint(lo, hi, shape, generator=self.g, device=DEV).to(dtype)

    def weight(self, n, k, bits, group, dtype):
        """Packed codes, all values of them, with scales and biases that give weights of
        about 1 / sqrt(k)."""
        wq = self.ints((n, k * bits // 32), -2 ** 31, 2 ** 31)
        top = 2 ** bits - 1
        s = self.uniform((n, k // group), 0.6, 1.4) * (3.4 / math.sqrt(k) / top)
        b = -s * top * self.uniform((n, k // group), 0.4, 0.6)
        return wq, s.to(dtype), b.to(dtype)

    def tokens(self, shape, v):
        """Token ids as text has them: id i about as often as 1 / (i + 3), shuffled."""
        u = torch.rand(shape, generator=self.g, device=DEV, dtype=torch.float64)
        i = ((v + 3) / 3.0) ** u * 3.0 - 3.0
        i = i.long().clamp(0, v - 1)
        return ((i * 7919 + 13) % v).to(torch.int32)

    def stream(self, shape, sigma, dtype):
        """Rows as a residual stream has them: a few channels far larger than the others."""
        t = self.normal(shape, sigma)
        t[:, 7::503] *= 30.0
        return t.to(dtype)


def prepare(case, seed):
    c, r = case, _Rand(seed)
    op, m, dt = c["op"], c["m"], DT[c["dtype"]]
    s = {"case": c}
    if op in ("loss", "loss_grad"):
        k, v = c["k"], c["v"]
        s["x"] = r.normal((m, k), 3.0, dt)          # logits of about 3
        s["w"] = r.weight(v, k, c["bits"], c["group"], dt)
        s["targets"] = r.tokens((m,), v)
        if m > 8:                                   # padding, without a target
            s["targets"][torch.rand((m,), generator=r.g, device=DEV) < 0.1] = -100
        if op == "loss_grad":
            # What the forward pass kept, and the mean over the rows with a target.
            z = s["x"].float() @ _dense(*s["w"], c["bits"], c["group"]).t()
            s["lse"] = _log_sum_exp(z)
            live = (s["targets"] >= 0).sum().clamp(min=1)
            s["dloss"] = (1.0 / live).expand(m).contiguous().float()
        return s
    d, st = c["d"], DT[c["stream"]]
    s["y"] = r.normal((m, d), 2.0, dt)
    mean = 1.0 - c["offset"]
    s["post"] = r.normal((d,), 0.2).add_(mean).to(dt) if c["post"] else None
    s["gate"] = r.normal((c["gates"], d), 0.5, dt) if c["gates"] else None
    s["weight"] = r.normal((d,), 0.2).add_(mean).to(dt) if c["pre"] else None
    s["factor"] = float(r.uniform((), 0.25, 1.0))
    s["x"] = r.stream((m, d), 4.0, st)
    if op == "norm_grad":
        s["s"] = _plain_norm(s)[0]                  # the stream that the forward pass wrote
        s["ds"] = r.normal((m, d), 0.1, st)
        s["da"] = r.normal((m, d), 0.1, dt) if c["pre"] else None
        del s["x"]                                  # not an input of the backward pass
    return s


# ------------------------------------------------------------------ the plain forms

def _codes(wq, bits):
    """Codes of packed rows, int32 [n, k]: each one's word and, where it crosses, the next."""
    n, words = wq.shape
    k = words * 32 // bits
    bit = torch.arange(k, device=wq.device) * bits
    at, sh = bit // 32, (bit % 32).to(torch.int64)
    w = wq.to(torch.int64) & 0xFFFFFFFF
    lo = w[:, at] >> sh
    hi = w[:, (at + 1).clamp(max=words - 1)] << (32 - sh)
    return (lo | hi) & (2 ** bits - 1)


def _spread(t, group):
    return t.float()[..., None].expand(*t.shape, group).reshape(*t.shape[:-1], -1)


def _dense(wq, scales, biases, bits, group):
    return _codes(wq, bits).float() * _spread(scales, group) + _spread(biases, group)


def _log_sum_exp(z):
    top = z.max(1).values
    return top + torch.log(torch.exp(z - top[:, None]).sum(1))


def _group_sums(wq, grad, bits, group):
    """Gradients of scales and biases from a dense weight's: sums over each group."""
    n, k = grad.shape
    ds = (grad * _codes(wq, bits).float()).reshape(n, k // group, group).sum(-1)
    return ds, grad.reshape(n, k // group, group).sum(-1)


def _plain_loss(s):
    c = s["case"]
    bits, group, dt = c["bits"], c["group"], DT[c["dtype"]]
    x, t = s["x"].float(), s["targets"].long()
    w = _dense(*s["w"], bits, group)
    z = x @ w.t()
    live = (t >= 0) & (t < c["v"])
    at = torch.where(live, t, torch.zeros_like(t))
    rows = torch.arange(c["m"], device=DEV)
    if c["op"] == "loss":
        lse = _log_sum_exp(z)
        return torch.where(live, lse - z[rows, at], torch.zeros_like(lse)), lse
    p = torch.exp(z - s["lse"][:, None])
    p[rows, at] -= 1.0
    dz = p * torch.where(live, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    ds, db = _group_sums(s["w"][0], dz.t() @ x, bits, group)
    return (dz @ w).to(dt), ds.to(dt), db.to(dt)


def _inverse_rms(v):
    return 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def _gate_rows(gate, m):
    """One row of the gate for each of the m rows."""
    g, d = gate.shape
    return gate.float()[:, None, :].expand(g, m // g, d).reshape(m, d)


def _plain_norm(s):
    """(s,) or (s, a)."""
    c = s["case"]
    t = s["y"].float()
    if s["post"] is not None:
        t = t * _inverse_rms(t) * (s["post"].float() + c["offset"])
    if s["gate"] is not None:
        t = t * _gate_rows(s["gate"], c["m"])
    v = s["x"].float() + s["factor"] * t
    if s["weight"] is None:
        return (v.to(DT[c["stream"]]),)
    a = v * _inverse_rms(v) * (s["weight"].float() + c["offset"])
    return v.to(DT[c["stream"]]), a.to(DT[c["dtype"]])


def _norm_back(v, u):
    """The gradient of v where u is that of v / rms(v)."""
    r = _inverse_rms(v)
    return r * u - v * r * r * r * (u * v).mean(-1, keepdim=True)


def _plain_norm_grad(s):
    """[dx, dy, dweight, dpost, dgate], those that there are."""
    c = s["case"]
    m, d, dt = c["m"], c["d"], DT[c["dtype"]]
    g = s["ds"].float()
    dweight = dpost = dgate = None
    if s["weight"] is not None:
        v, da = s["s"].float(), s["da"].float()
        dweight = (da * v * _inverse_rms(v)).sum(0)
        g = g + _norm_back(v, da * (s["weight"].float() + c["offset"]))
    y = s["y"].float()
    n = y * _inverse_rms(y) if s["post"] is not None else y
    t = n * (s["post"].float() + c["offset"]) if s["post"] is not None else n
    dt_ = s["factor"] * g
    if s["gate"] is not None:
        rows = s["gate"].shape[0]
        dgate = (t * dt_).reshape(rows, m // rows, d).sum(1)
        dt_ = dt_ * _gate_rows(s["gate"], m)
    dy = dt_
    if s["post"] is not None:
        dpost = (dt_ * n).sum(0)
        dy = _norm_back(y, dt_ * (s["post"].float() + c["offset"]))
    return [g.to(DT[c["stream"]]), dy.to(dt)] + [t.to(dt) for t in (dweight, dpost, dgate) if t is not None]


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op in ("loss", "loss_grad"):
            return _plain_loss(s)
        return _plain_norm(s) if op == "norm" else _plain_norm_grad(s)
    import weight_only_quantized_qgemv_amd as qp
    if op == "loss":
        return qp.qcross_entropy(s["x"], s["targets"], *s["w"], c["bits"], c["group"])
    if op == "loss_grad":
        return qp.qcross_entropy_backward(s["x"], s["targets"], s["lse"], s["dloss"], *s["w"], c["bits"], c["group"])
    parts = {"y": s["y"], "weight": s["weight"], "post_weight": s["post"], "gate": s["gate"], "scale": s["factor"],
             "offset": c["offset"], "eps": EPS}
    if op == "norm":
        out = qp.qblock_norm(s["x"], **parts)
        return out if s["weight"] is not None else out[:1]
    return [t for t in qp.qblock_norm_backward(s["s"], da=s["da"], ds=s["ds"], **parts) if t is not None]


def work(case):
    """Each input read once, each output written once, the products' multiplications and
    additions."""
    c = case
    m, e = c["m"], 2 if c["dtype"] != "f32" else 4
    if c["op"] in ("loss", "loss_grad"):
        k, v = c["k"], c["v"]
        params = 2 * v * (k // c["group"]) * e
        w = v * k * c["bits"] // 8 + params
        if c["op"] == "loss":
            return {"bytes": w + m * k * e + 12 * m, "flops": 2 * m * k * v}
        return {"bytes": w + 2 * m * k * e + 12 * m + params, "flops": 6 * m * k * v}
    d, st = c["d"], 2 if c["stream"] != "f32" else 4
    small = e * d * (int(c["post"]) + c["gates"] + int(c["pre"]))
    rows = 2 * st + e + (e if c["pre"] else 0)     # x, s, y, a
    if c["op"] == "norm_grad":                      # ds, dx, y, dy, and da and s
        rows = 2 * st + 2 * e + (st + e if c["pre"] else 0)
        small *= 2
    return {"bytes": rows * m * d + small, "flops": 0}


# ------------------------------------------------------------------ 64 bits

def _dense64(w, bits, group):
    """The weight from the rows' single bits."""
    wq, s, b = w
    n, words = wq.shape
    bit = torch.arange(32, device=wq.device, dtype=torch.int32)
    stream = ((wq[:, :, None] >> bit) & 1).to(torch.uint8).reshape(n, -1, bits)
    q = torch.zeros((n, stream.shape[1]), device=wq.device, dtype=torch.float64)
    for i in range(bits):
        q += stream[:, :, i].double() * float(2 ** i)
    q = q.reshape(n, -1, group)
    return (q * s.double()[:, :, None] + b.double()[:, :, None]).reshape(n, -1), q


def _exact_loss(s):
    c = s["case"]
    bits, group, v = c["bits"], c["group"], c["v"]
    x, t = s["x"].double(), s["targets"].long()
    w, q = _dense64(s["w"], bits, group)
    z = torch.nn.functional.linear(x, w)
    live = ((t >= 0) & (t < v)).double()
    at = t.clamp(0, v - 1)[:, None]
    if c["op"] == "loss":
        lse = torch.logsumexp(z, 1)
        return (lse - z.gather(1, at)[:, 0]) * live, lse
    z.sub_(s["lse"].double()[:, None]).exp_()
    z.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    z.mul_((live * s["dloss"].double())[:, None])
    dx = torch.mm(z, w)
    grad = torch.mm(z.t(), x).reshape(q.shape)
    return dx, (grad * q).sum(-1), grad.sum(-1)


def _rms64(v):
    return torch.sqrt(torch.linalg.vector_norm(v, dim=-1, keepdim=True) ** 2 / v.shape[-1] + EPS)


def _exact_norm(s):
    c = s["case"]
    m, d = c["m"], c["d"]
    y = s["y"].double()
    one = torch.ones((1, d), device=DEV, dtype=torch.float64)
    gate = one if s["gate"] is None else s["gate"].double()
    gate = gate.repeat_interleave(m // gate.shape[0], 0) * s["factor"]
    post = None if s["post"] is None else s["post"].double() + c["offset"]
    weight = None if s["weight"] is None else s["weight"].double() + c["offset"]
    n = y if post is None else y / _rms64(y)
    t = n if post is None else n * post
    if c["op"] == "norm":
        v = s["x"].double() + gate * t
        return (v,) if weight is None else (v, weight * v / _rms64(v))
    g = s["ds"].double()
    out = []
    if weight is not None:
        v, da = s["s"].double(), s["da"].double()
        h = v / _rms64(v)
        out.append((da * h).sum(0))
        u = da * weight
        g = g + (u - h * (u * h).sum(-1, keepdim=True) / d) / _rms64(v)
    u = g * gate
    dy = u
    if post is not None:
        out.append((u * n).sum(0))
        u = u * post
        dy = (u - n * (u * n).sum(-1, keepdim=True) / d) / _rms64(y)
    if s["gate"] is not None:
        rows = s["gate"].shape[0]
        out.append((g * t * s["factor"]).reshape(rows, m // rows, d).sum(1))
    return [g, dy] + out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_loss(s) if case["op"] in ("loss", "loss_grad") else _exact_norm(s)
