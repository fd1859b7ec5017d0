"""The language-model operators around the quantized products, as measured cases.

Four operators, each with a plain form in elementary torch operations (fp32, rounded
once at the end) and the library's call:

- ``ffn`` / ``ffn_grad``: the dense gated feed-forward block over packed weights,
  y = (act(x Wg^T) * (x Wu^T)) Wd^T, and its gradients with respect to the input and to
  the groups' scales and biases of the three weights (the codes are integers and stay);
- ``linear_grad``: the gradients of one quantized linear layer, y = x W^T;
- ``embed`` / ``embed_grad``: lookup of packed table rows with a factor, and the gradient
  of the table's scales and biases, summed over the tokens of each row;
- ``logits``: repetition, frequency and presence penalties from each sequence's tokens,
  a sparse bias and a bit mask of allowed tokens, over a batch of logit rows.

W[n, k] = q[n, k] * scale[n, k // group] + bias[n, k // group], code k of a row at bit
k * bits of the row's little-endian 32-bit words.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def _ffn(name, op, m, d, f, bits, group, dtype, act, train=False):
    c = {"name": name, "op": op, "m": m, "d": d, "f": f, "bits": bits, "group": group,
         "dtype": dtype, "act": act}
    if op == "ffn":
        c["train"] = train
    return c


def listed():
    return [
        # One new token through a block: the weights are read once, nothing else counts.
        _ffn("ffn_decode_1", "ffn", 1, 4096, 14336, 4, 64, "bf16", "silu"),
        # A small batch of decoding sequences, an odd number of them, at 8 bits.
        _ffn("ffn_decode_12", "ffn", 12, 2048, 5632, 8, 32, "f16", "gelu_tanh"),
        # The forward pass of a training step, keeping what its backward pass needs.
        _ffn("ffn_train_2048", "ffn", 2048, 4096, 14336, 4, 64, "bf16", "silu", True),
        # A short odd sequence's backward pass on a small model, 6-bit codes across words.
        _ffn("ffn_grad_77", "ffn_grad", 77, 1024, 2816, 6, 32, "f16", "gelu_tanh"),
        # The backward pass of a training step.
        _ffn("ffn_grad_2048", "ffn_grad", 2048, 4096, 14336, 4, 64, "bf16", "silu"),
        # The output head's backward pass over a packed batch of an uneven length.
        {"name": "linear_grad_1000", "op": "linear_grad", "m": 1000, "k": 4096, "n": 32000,
         "bits": 8, "group": 64, "dtype": "bf16"},
        # A small layer trained in fp32.
        {"name": "linear_grad_130_f32", "op": "linear_grad", "m": 130, "k": 768, "n": 2048,
         "bits": 3, "group": 32, "dtype": "f32"},
        # One decoded token per sequence of a small batch.
        {"name": "embed_7", "op": "embed", "t": 7, "v": 32000, "k": 4096, "bits": 4, "group": 64,
         "dtype": "bf16", "factor": 1.0},
        # A packed batch of prompts, with the embedding's factor.
        {"name": "embed_16384", "op": "embed", "t": 16384, "v": 131072, "k": 2048, "bits": 8,
         "group": 32, "dtype": "f16", "factor": 45.25},
        # A training step's tokens: a few ids very often, most of them once or never.
        {"name": "embed_grad_8192", "op": "embed_grad", "t": 8192, "v": 32000, "k": 4096,
         "bits": 4, "group": 64, "dtype": "bf16", "factor": 1.0},
        # One sequence sampling with penalties and no mask.
        {"name": "logits_1", "op": "logits", "rows": 1, "v": 32000, "pad": 0, "hist": 700,
         "bias": 12, "mask": False, "dtype": "f32"},
        # A serving batch with every control, rows padded, an odd vocabulary.
        {"name": "logits_64", "op": "logits", "rows": 64, "v": 131071, "pad": 65, "hist": 4000,
         "bias": 300, "mask": True, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n == 3072 else n


def _log_size(rng, lo, hi, step):
    n = max(1, _log_int(rng, lo, hi) // step) * step
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(["ffn", "ffn_grad", "linear_grad", "embed", "embed_grad", "logits"])
    bits, group = rng.choice([2, 3, 4, 4, 6, 8]), rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("ffn", "ffn_grad"):
        c = {"op": op, "m": _log_int(rng, 1, 2048), "d": _log_size(rng, 128, 4096, group),
             "f": _log_size(rng, 256, 14336, group), "bits": bits, "group": group, "dtype": dtype,
             "act": rng.choice(["silu", "gelu_tanh"])}
        if op == "ffn":
            c["train"] = rng.choice([False, True])
        return c
    if op == "linear_grad":
        return {"op": op, "m": _log_int(rng, 1, 2048), "k": _log_size(rng, 128, 4096, group),
                "n": _log_int(rng, 100, 32000), "bits": bits, "group": group, "dtype": dtype}
    if op in ("embed", "embed_grad"):
        return {"op": op, "t": _log_int(rng, 1, 16384), "v": _log_int(rng, 1000, 131072),
                "k": _log_size(rng, 128, 4096, group), "bits": bits, "group": group,
                "dtype": dtype, "factor": rng.choice([1.0, 16.0, 45.25])}
    return {"op": op, "rows": _log_int(rng, 1, 128), "v": _log_int(rng, 1000, 131072),
            "pad": rng.choice([0, 1, 64]), "hist": _log_int(rng, 1, 4096),
            "bias": rng.choice([0, 12, 300]), "mask": rng.choice([False, True]), "dtype": dtype}


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


def prepare(case, seed):
    c, r = case, _Rand(seed)
    op = c["op"]
    s = {"case": c}
    if op == "logits":
        rows, v = c["rows"], c["v"]
        s["logits"] = r.normal((rows, v + c["pad"]), 4.0, DT[c["dtype"]])[:, :v]
        # Sequences of different lengths, one of them without a token yet when there are several.
        lens = r.ints((rows,), 1 + c["hist"] // 4, c["hist"] + 1)
        if rows > 2:
            lens[1] = 0
        s["offsets"] = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
        total = int(s["offsets"][-1])
        s["history"] = r.tokens((total,), v)
        s["prompt_lens"] = (lens * r.uniform((rows,), 0.0, 1.0)).to(torch.int32)
        s["repetition"] = r.uniform((rows,), 1.0, 1.5)
        s["frequency"] = r.uniform((rows,), 0.0, 0.8)
        s["presence"] = r.uniform((rows,), -0.2, 0.8)
        s["bias"] = None
        if c["bias"]:
            # Distinct tokens of a row: a random start, a step coprime to any count below v.
            n = c["bias"]
            start = r.ints((rows, 1), 0, v, torch.int64)
            ids = (start + torch.arange(n, device=DEV) * (v // n)) % v
            s["bias"] = (ids.to(torch.int32).reshape(-1), r.normal((rows * n,), 3.0),
                         (torch.arange(rows + 1, device=DEV) * n).to(torch.int32))
        s["mask"] = r.ints((rows, (v + 31) // 32), -2 ** 31, 2 ** 31) if c["mask"] else None
        return s
    dt = DT[c["dtype"]]
    bits, group = c["bits"], c["group"]
    if op in ("ffn", "ffn_grad"):
        m, d, f = c["m"], c["d"], c["f"]
        s["x"] = r.normal((m, d), 1.0, dt)
        s["gate"], s["up"] = (r.weight(f, d, bits, group, dt) for _ in range(2))
        s["down"] = r.weight(d, f, bits, group, dt)
        if op == "ffn_grad":
            s["dy"] = r.normal((m, d), 0.1, dt)
            # What the forward pass kept.
            s["saved"] = torch.stack([s["x"].float() @ _dense(*s[w], bits, group).t()
                                      for w in ("gate", "up")]).to(dt)
    elif op == "linear_grad":
        s["x"], s["dy"] = r.normal((c["m"], c["k"]), 1.0, dt), r.normal((c["m"], c["n"]), 0.1, dt)
        s["w"] = r.weight(c["n"], c["k"], bits, group, dt)
    else:
        s["ids"] = r.tokens((c["t"],), c["v"])
        s["table"] = r.weight(c["v"], c["k"], bits, group, dt)
        if op == "embed_grad":
            s["dout"] = r.normal((c["t"], c["k"]), 0.1, dt)
    return s


# ------------------------------------------------------------------ the plain forms

def _codes(wq, bits):
    """Codes of packed rows, int64 [n, k]: each one's word and, where it crosses, the next."""
    n, words = wq.shape
    k = words * 32 // bits
    bit = torch.arange(k, device=wq.device) * bits
    at, sh = bit // 32, bit % 32
    w = wq.to(torch.int64) & 0xFFFFFFFF
    lo = w[:, at] >> sh
    hi = w[:, (at + 1).clamp(max=words - 1)] << (32 - sh)
    return (lo | hi) & (2 ** bits - 1)


def _spread(t, group):
    return t.float()[..., None].expand(*t.shape, group).reshape(*t.shape[:-1], -1)


def _dense(wq, scales, biases, bits, group):
    return _codes(wq, bits).float() * _spread(scales, group) + _spread(biases, group)


def _act(z, act):
    """The activation and its derivative."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return z * sig, sig * (1 + z * (1 - sig))
    a, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(a * (z + b * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * b * z * z)


def _group_sums(wq, grad, bits, group):
    """Gradients of scales and biases from a dense weight's: sums over each group."""
    n, k = grad.shape
    ds = (grad * _codes(wq, bits).float()).reshape(n, k // group, group).sum(-1)
    return ds, grad.reshape(n, k // group, group).sum(-1)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "logits":
        return _plain_logits(s)
    bits, group, dt = c["bits"], c["group"], DT[c["dtype"]]
    if op == "ffn":
        x = s["x"].float()
        g = x @ _dense(*s["gate"], bits, group).t()
        u = x @ _dense(*s["up"], bits, group).t()
        y = (_act(g, c["act"])[0] * u) @ _dense(*s["down"], bits, group).t()
        return (y.to(dt), torch.stack([g, u]).to(dt)) if c["train"] else y.to(dt)
    if op == "ffn_grad":
        x, dy, (g, u) = s["x"].float(), s["dy"].float(), s["saved"].float()
        a, da = _act(g, c["act"])
        dh = dy @ _dense(*s["down"], bits, group)
        dg, du = dh * u * da, dh * a
        dx = dg @ _dense(*s["gate"], bits, group) + du @ _dense(*s["up"], bits, group)
        grads = [_group_sums(s[w][0], dz.t() @ z, bits, group)
                 for w, dz, z in (("gate", dg, x), ("up", du, x), ("down", dy, a * u))]
        return dx.to(dt), [t.to(dt) for p in grads for t in p]
    if op == "linear_grad":
        x, dy = s["x"].float(), s["dy"].float()
        dx = dy @ _dense(*s["w"], bits, group)
        ds, db = _group_sums(s["w"][0], dy.t() @ x, bits, group)
        return dx.to(dt), ds.to(dt), db.to(dt)
    wq, scales, biases = s["table"]
    at = s["ids"].long()
    if op == "embed":
        return (_dense(wq[at], scales[at], biases[at], bits, group) * c["factor"]).to(dt)
    # The rows' gradients by sorted tokens: runs of equal ids as differences of running sums
    # would lose precision, so each row of the table is summed by index.
    grad = torch.zeros((c["v"], c["k"]), device=DEV)
    grad.index_add_(0, at, s["dout"].float())
    ds, db = _group_sums(wq, grad, bits, group)
    return (ds * c["factor"]).to(dt), (db * c["factor"]).to(dt)


def _plain_logits(s):
    z = s["logits"].float()
    rows, v = z.shape
    off, hist = s["offsets"].long(), s["history"].long()
    at = torch.arange(hist.numel(), device=DEV)
    row = torch.searchsorted(off[1:].contiguous(), at, right=True)
    made = at - off[row] >= s["prompt_lens"].long()[row]
    flat = row * v + hist
    seen = torch.zeros(rows * v, device=DEV).index_fill_(0, flat, 1.0).reshape(rows, v) > 0
    count = torch.zeros(rows * v, device=DEV, dtype=torch.int32)
    count = count.scatter_add_(0, flat, made.int()).reshape(rows, v).float()
    rep = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias"] is not None:
        ids, values, boff = s["bias"]
        j = torch.arange(ids.numel(), device=DEV)
        brow = torch.searchsorted(boff[1:].long().contiguous(), j, right=True)
        z = z + torch.zeros(rows * v, device=DEV).scatter_(0, brow * v + ids.long(), values).reshape(rows, v)
    if s["mask"] is not None:
        j = torch.arange(v, device=DEV)
        allowed = (s["mask"].long()[:, j // 32] >> (j % 32)) & 1
        z = torch.where(allowed > 0, z, torch.full_like(z, -math.inf))
    return z.to(s["logits"].dtype)


# ------------------------------------------------------------------ one pass

def run(state):
    if not own:
        return _plain(state)
    import weight_only_quantized_qgemv_amd as qp
    s, c = state, state["case"]
    op = c["op"]
    if op == "logits":
        return qp.qlogits_adjust(s["logits"], history=s["history"], offsets=s["offsets"],
                                 prompt_lens=s["prompt_lens"], repetition=s["repetition"],
                                 frequency=s["frequency"], presence=s["presence"], bias=s["bias"],
                                 mask=s["mask"])
    bits, group = c["bits"], c["group"]
    if op == "ffn":
        if not c["train"]:
            return qp.qffn(s["x"], s["gate"], s["up"], s["down"], bits, group, act=c["act"])
        saved = torch.empty((2, c["m"], c["f"]), dtype=s["x"].dtype, device=s["x"].device)
        return qp.qffn(s["x"], s["gate"], s["up"], s["down"], bits, group, act=c["act"],
                       saved=saved), saved
    if op == "ffn_grad":
        dx, *grads = qp.qffn_backward(s["x"], s["dy"], s["saved"], s["gate"], s["up"], s["down"],
                                      bits, group, act=c["act"])
        return dx, [t for p in grads for t in p]
    if op == "linear_grad":
        return qp.qmatmul_backward(s["x"], s["dy"], *s["w"], bits, group)
    if op == "embed":
        return qp.qembedding(s["ids"], *s["table"], bits, group, factor=c["factor"])
    return qp.qembedding_backward(s["ids"], s["dout"], s["table"][0], bits, group,
                                  factor=c["factor"])


def work(case):
    """Each input read once, each output written once, the products' multiplications and
    additions."""
    c = case
    op, e = c["op"], 2 if c["dtype"] != "f32" else 4
    if op == "logits":
        n = c["rows"] * c["v"]
        hist = c["rows"] * c["hist"] * 5 // 8
        return {"bytes": 2 * n * e + 4 * hist + 8 * c["rows"] * c["bias"]
                + (n // 8 if c["mask"] else 0), "flops": 0}

    def packed(n, k):
        return n * k * c["bits"] // 8 + 2 * n * (k // c["group"]) * e

    def params(n, k):
        return 2 * n * (k // c["group"]) * e

    if op in ("ffn", "ffn_grad"):
        m, d, f = c["m"], c["d"], c["f"]
        w = 2 * packed(f, d) + packed(d, f)
        if op == "ffn":
            return {"bytes": w + 2 * m * d * e + (2 * m * f * e if c["train"] else 0),
                    "flops": 6 * m * d * f}
        return {"bytes": w + 3 * m * d * e + 2 * m * f * e + 2 * params(f, d) + params(d, f),
                "flops": 12 * m * d * f}
    if op == "linear_grad":
        m, k, n = c["m"], c["k"], c["n"]
        return {"bytes": packed(n, k) + (2 * m * k + m * n) * e + params(n, k),
                "flops": 4 * m * n * k}
    t, v, k = c["t"], c["v"], c["k"]
    if op == "embed":
        return {"bytes": 4 * t + packed(min(t, v), k) + t * k * e, "flops": 3 * t * k}
    rows = min(t, v)
    return {"bytes": 4 * t + t * k * e + rows * k * c["bits"] // 8 + params(v, k),
            "flops": 3 * t * k}


# ------------------------------------------------------------------ 64 bits

def _codes64(wq, bits):
    """The codes from the rows' single bits."""
    n, words = wq.shape
    bit = torch.arange(32, device=wq.device, dtype=torch.int32)
    stream = ((wq[:, :, None] >> bit) & 1).to(torch.uint8).reshape(n, -1, bits)
    weight = (2 ** torch.arange(bits, device=wq.device)).double()
    out = torch.zeros((n, stream.shape[1]), device=wq.device, dtype=torch.float64)
    for i in range(bits):
        out += stream[:, :, i].double() * weight[i]
    return out


def _dense64(w, bits, group):
    wq, s, b = w
    q = _codes64(wq, bits)
    n, k = q.shape
    q = q.reshape(n, k // group, group)
    return (q * s.double()[:, :, None] + b.double()[:, :, None]).reshape(n, k)


def _act64(z, act):
    if act == "silu":
        sig = torch.sigmoid(z)
        return z * sig, sig + z * sig * torch.sigmoid(-z)
    # 0.5 (1 + tanh y) = sigmoid(2 y)
    a = 2 * math.sqrt(2 / math.pi)
    y = a * (z + 0.044715 * z ** 3)
    sig = torch.sigmoid(y)
    return z * sig, sig + z * sig * torch.sigmoid(-y) * a * (1 + 3 * 0.044715 * z ** 2)


def _param_grads64(wq, left, right, bits, group, factor=1.0):
    """(dscales, dbiases) of the weight whose dense gradient is left^T right."""
    n, k = left.shape[1], right.shape[1]
    grad = (left.t() @ right).reshape(n, k // group, group)
    q = _codes64(wq, bits).reshape(n, k // group, group)
    return [factor * (grad * q).sum(-1), factor * grad.sum(-1)]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    op = c["op"]
    if op == "logits":
        return _exact_logits(s)
    bits, group = c["bits"], c["group"]
    if op == "ffn":
        x = s["x"].double()
        g, u = (torch.nn.functional.linear(x, _dense64(s[w], bits, group)) for w in ("gate", "up"))
        y = torch.nn.functional.linear(_act64(g, c["act"])[0] * u, _dense64(s["down"], bits, group))
        return (y, torch.stack([g, u])) if c["train"] else y
    if op == "ffn_grad":
        x, dy, g, u = s["x"].double(), s["dy"].double(), s["saved"][0].double(), s["saved"][1].double()
        a, da = _act64(g, c["act"])
        dh = torch.mm(dy, _dense64(s["down"], bits, group))
        dg, du = dh * u * da, dh * a
        dx = torch.mm(dg, _dense64(s["gate"], bits, group))
        dx += torch.mm(du, _dense64(s["up"], bits, group))
        return dx, (_param_grads64(s["gate"][0], dg, x, bits, group)
                    + _param_grads64(s["up"][0], du, x, bits, group)
                    + _param_grads64(s["down"][0], dy, a * u, bits, group))
    if op == "linear_grad":
        x, dy = s["x"].double(), s["dy"].double()
        ds, db = _param_grads64(s["w"][0], dy, x, bits, group)
        return torch.mm(dy, _dense64(s["w"], bits, group)), ds, db
    ids = s["ids"].long()
    if op == "embed":
        w = tuple(t[ids] for t in s["table"])
        return _dense64(w, bits, group) * c["factor"]
    # Only the rows that occur have a gradient.
    seen, back = torch.unique(ids, return_inverse=True)
    grad = torch.zeros((seen.numel(), c["k"]), device=DEV, dtype=torch.float64)
    grad.index_add_(0, back, s["dout"].double() * c["factor"])
    q = _codes64(s["table"][0][seen], bits)
    shape = (seen.numel(), c["k"] // group, group)
    out = []
    for t in ((grad * q).reshape(shape).sum(-1), grad.reshape(shape).sum(-1)):
        full = torch.zeros((c["v"], c["k"] // group), device=DEV, dtype=torch.float64)
        full[seen] = t
        out.append(full)
    return tuple(out)


def _exact_logits(s):
    z = s["logits"].double().clone()
    rows, v = z.shape
    off = s["offsets"].tolist()
    for r in range(rows):
        h = s["history"][off[r]:off[r + 1]].long()
        made = h[int(s["prompt_lens"][r]):]
        rep, freq, pres = (float(s[n][r]) for n in ("repetition", "frequency", "presence"))
        seen = torch.unique(h)
        w = z[r, seen]
        z[r, seen] = torch.where(w > 0, w / rep, w * rep)
        tok, cnt = torch.unique(made, return_counts=True)
        z[r, tok] -= freq * cnt.double() + pres
        if s["bias"] is not None:
            ids, values, boff = s["bias"]
            b0, b1 = int(boff[r]), int(boff[r + 1])
            z[r, ids[b0:b1].long()] += values[b0:b1].double()
    if s["mask"] is not None:
        bit = torch.arange(32, device=DEV, dtype=torch.int32)
        allowed = ((s["mask"][:, :, None] >> bit) & 1).reshape(rows, -1)[:, :v]
        z[allowed == 0] = -math.inf
    return z
