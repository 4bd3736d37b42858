"""Timed cases of a gated MLP's training step: the gated product (both projections, the activation
and their product), its backward product, and the orthogonalised update of its weights by
Newton-Schulz products.

`own` chooses between the plain form (elementary torch operations in 32 bits, rounded once) and
the library's calls. `exact` gives the same outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
STEP = (3.4445, -4.7750, 2.0315)  # coefficients of one Newton-Schulz step, the library's default
EPS = 1e-7


# ------------------------------------------------------------------------------ cases
def _glu(name, m, n, k, act, *, ta=False, tb=True, keep=False):
    return dict(name=name, op="glu", m=m, n=n, k=k, act=act, ta=ta, tb=tb, keep=keep)


def _dglu(name, m, n, k, act, *, ta=False, tb=False, hidden=True):
    return dict(name=name, op="dglu", m=m, n=n, k=k, act=act, ta=ta, tb=tb, hidden=hidden)


def _orth(name, m, n, *, x="bf16", steps=5, beta=0.0):
    return dict(name=name, op="orthogonalize", m=m, n=n, x=x, steps=steps, beta=beta)


def listed():
    return [
        # one token of a served model through the gate and the up projection
        _glu("glu_1x4096x4096_silu", 1, 4096, 4096, "silu"),
        # a small batch of served tokens of a larger model
        _glu("glu_24x16384x5120_silu", 24, 16384, 5120, "silu"),
        # training forward, both pre-activations kept for the backward pass
        _glu("glu_4096x16384x4096_silu_kept", 4096, 16384, 4096, "silu", keep=True),
        # odd sizes, weights stored [k, n]: rows of the outputs end off a 16-byte boundary
        _glu("glu_1111x2162x1000_gelu", 1111, 2162, 1000, "gelu", tb=False),
        # training backward through the down projection and the gate, the activation computed again
        _dglu("dglu_4096x16384x4096_silu", 4096, 16384, 4096, "silu"),
        # the same for a short ragged batch of a small model
        _dglu("dglu_777x1320x520_gelu_tanh", 777, 1320, 520, "gelu_tanh"),
        # the update of a small model's square projection, and of one head's: launch latency counts
        _orth("orth_1024x1024", 1024, 1024),
        _orth("orth_128x128", 128, 128),
        # of an up projection stored [n, k] and its down projection, BF16 momentum
        _orth("orth_16384x4096", 16384, 4096),
        _orth("orth_4096x4096", 4096, 4096),
        # odd sizes, FP32 momentum, added to the decayed weights
        _orth("orth_1000x2162_f32_update", 1000, 2162, x="f32", beta=0.99),
    ]


_MOST_PRODUCT = 4096 * 16384 * 4096              # m n k of the largest listed backward product
_MOST_ORTH = 3 * 4096 * 4096 * 16384 + 4096 ** 3  # flops of one step of the largest listed update


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("glu", "glu", "dglu", "orthogonalize", "orthogonalize"))
    if op == "orthogonalize":
        while True:
            m, n = _log_int(rng, 16, 16384), _log_int(rng, 16, 16384)
            s, long = min(m, n), max(m, n)
            if 3 * s * s * long + s ** 3 <= _MOST_ORTH // 4:
                break
        c = _orth("", m, n, x=rng.choice(("bf16", "f32")), steps=rng.choice((3, 5, 5, 5)), beta=rng.choice((0.0, 0.0, 0.99)))
    else:
        act = rng.choice(ACTS)
        while True:
            m, n, k = _log_int(rng, 1, 8192), _log_int(rng, 64, 16384), _log_int(rng, 64, 8192)
            if m * n * k <= _MOST_PRODUCT // 4 and m * n <= 4096 * 16384 // 2:
                break
        if op == "glu":
            c = _glu("", m, n, k, act, ta=rng.random() < 0.15, tb=rng.random() < 0.7, keep=rng.random() < 0.5)
        else:
            c = _dglu("", m, n, k, act, ta=rng.random() < 0.15, tb=rng.random() < 0.3, hidden=rng.random() < 0.7)
    del c["name"]
    return c


# ------------------------------------------------------------------------------ inputs
def _rows16(rows, cols, dtype=torch.bfloat16):
    """[rows, cols] whose rows start on 16-byte boundaries, as the library asks of its callers."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty((rows, -(-cols // per) * per), dtype=dtype, device="cuda")[:, :cols]


def _normal(gen, rows, cols, std, dtype=torch.bfloat16):
    out = _rows16(rows, cols, dtype)
    out.copy_(torch.randn((rows, cols), generator=gen, device="cuda") * std)
    return out


def _momentum(gen, rows, cols, dtype):
    """A weight's averaged gradient: directions of falling size over a floor of noise, small in absolute terms."""
    rank = max(1, min(rows, cols, 256) // 2)
    falling = torch.arange(1, rank + 1, device="cuda").float().pow(-0.7)
    left = torch.randn((rows, rank), generator=gen, device="cuda") * falling
    right = torch.randn((rank, cols), generator=gen, device="cuda")
    noise = torch.randn((rows, cols), generator=gen, device="cuda")
    out = _rows16(rows, cols, dtype)
    out.copy_((left @ right + 0.5 * noise) * 1e-4)
    return out


class _State:
    def __init__(self, case, seed):
        self.case = c = case
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        op, m, n = c["op"], c["m"], c["n"]
        if op == "glu":
            # activations of unit size, weights that keep the products' size
            k = c["k"]
            self.A = _normal(g, *((k, m) if c["ta"] else (m, k)), 1.0)
            shape = (n, k) if c["tb"] else (k, n)
            self.Wg, self.Wu = _normal(g, *shape, 1.0 / math.sqrt(k)), _normal(g, *shape, 1.0 / math.sqrt(k))
            self.H = _rows16(m, n)
            self.G, self.U = (_rows16(m, n), _rows16(m, n)) if c["keep"] else (None, None)
        elif op == "dglu":
            k = c["k"]
            self.A = _normal(g, *((k, m) if c["ta"] else (m, k)), 0.01)
            self.B = _normal(g, *((n, k) if c["tb"] else (k, n)), 1.0 / math.sqrt(k))
            self.G, self.U = _normal(g, m, n, 1.0), _normal(g, m, n, 1.0)
            self.dG, self.dU = _rows16(m, n), _rows16(m, n)
            self.H = _rows16(m, n) if c["hidden"] else None
        else:
            self.X = _momentum(g, m, n, torch.float32 if c["x"] == "f32" else torch.bfloat16)
            # the update's size follows the longer side; with beta the weights lie in C
            self.alpha = 1.0 if c["beta"] == 0.0 else -0.02 * math.sqrt(max(1.0, m / n))
            self.C = _normal(g, m, n, 1.0 / math.sqrt(n))
            # what a program keeps for such calls (a few copies of X and of the square of its shorter side)
            s = min(m, n) + 8
            self.workspace = torch.empty(8 * (m + 8) * (n + 8) + 8 * s * s + (32 << 20), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    return _State(case, seed)


# ------------------------------------------------------------------------------ plain form
def _activate(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _derivative(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def _plain(s):
    c = s.case
    if c["op"] == "glu":
        a = s.A.float().t() if c["ta"] else s.A.float()
        wg, wu = (w.float().t() if c["tb"] else w.float() for w in (s.Wg, s.Wu))
        gate, up = a @ wg, a @ wu
        h = (_activate(gate, c["act"]) * up).to(s.H.dtype)
        return (h, gate.to(s.G.dtype), up.to(s.U.dtype)) if c["keep"] else h
    if c["op"] == "dglu":
        dh = (s.A.float().t() if c["ta"] else s.A.float()) @ (s.B.float().t() if c["tb"] else s.B.float())
        gate, up = s.G.float(), s.U.float()
        value = _activate(gate, c["act"])
        out = ((dh * up * _derivative(gate, c["act"])).to(s.dG.dtype), (dh * value).to(s.dU.dtype))
        return out + ((value * up).to(s.H.dtype),) if c["hidden"] else out
    x = s.X.float()
    x = x / (x.norm() + EPS)
    a, b, q = STEP
    wide = c["m"] <= c["n"]
    for _ in range(c["steps"]):
        gram = x @ x.t() if wide else x.t() @ x
        poly = b * gram + q * (gram @ gram)
        x = a * x + (poly @ x if wide else x @ poly)
    out = s.alpha * x
    if c["beta"] != 0.0:
        out = out + c["beta"] * s.C.float()
    return s.C.copy_(out)


# ------------------------------------------------------------------------------ one pass
def run(s):
    if not own:
        return _plain(s)
    import blas3_tensor_core_gb300 as bm
    c = s.case
    if c["op"] == "glu":
        bm.gemm_glu(s.A, s.Wg, s.Wu, s.H, act=c["act"], gate=s.G, up=s.U, transA=c["ta"], transB=c["tb"])
        return (s.H, s.G, s.U) if c["keep"] else s.H
    if c["op"] == "dglu":
        bm.gemm_dglu(s.A, s.B, s.G, s.U, s.dG, s.dU, act=c["act"], hidden=s.H, transA=c["ta"], transB=c["tb"])
        return (s.dG, s.dU, s.H) if c["hidden"] else (s.dG, s.dU)
    return bm.orthogonalize(s.X, s.C, alpha=s.alpha, beta=c["beta"], steps=c["steps"], eps=EPS, workspace=s.workspace)


def work(case):
    c = case
    mn = c["m"] * c["n"]
    if c["op"] == "glu":
        return {"bytes": 2 * c["k"] * (c["m"] + 2 * c["n"]) + 2 * mn * (3 if c["keep"] else 1), "flops": 4 * mn * c["k"]}
    if c["op"] == "dglu":
        return {"bytes": 2 * c["k"] * (c["m"] + c["n"]) + 2 * mn * (5 if c["hidden"] else 4), "flops": 2 * mn * c["k"]}
    # the Gram matrix and its square are symmetric: one triangle of each
    s, long = min(c["m"], c["n"]), max(c["m"], c["n"])
    return {"bytes": mn * ((4 if c["x"] == "f32" else 2) + (2 if c["beta"] == 0.0 else 4)),
            "flops": c["steps"] * (3 * s * s * long + s ** 3)}


# ------------------------------------------------------------------------------ 64 bits
def _exact_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1 + torch.exp(-z))


def _exact_slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        p = 1 / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        return p + z * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def exact(case, seed):
    c, s = case, _State(case, seed)
    if c["op"] == "glu":
        a = s.A.double().t() if c["ta"] else s.A.double()
        gate = torch.mm(a, s.Wg.double().t() if c["tb"] else s.Wg.double())
        up = torch.mm(a, s.Wu.double().t() if c["tb"] else s.Wu.double())
        h = _exact_act(gate, c["act"]).mul_(up)
        return (h, gate, up) if c["keep"] else h
    if c["op"] == "dglu":
        dh = torch.mm(s.A.double().t() if c["ta"] else s.A.double(), s.B.double().t() if c["tb"] else s.B.double())
        gate, up = s.G.double(), s.U.double()
        h = _exact_act(gate, c["act"])
        out = (_exact_slope(gate, c["act"]) * up * dh, h * dh)
        return out + (h * up,) if c["hidden"] else out
    # x (a I + b x'x + c (x'x)^2) over the shorter side, on a matrix with the short side last
    tall = c["m"] >= c["n"]
    x = s.X.double() if tall else s.X.double().t().contiguous()
    x = x / (torch.sqrt((x * x).sum()) + EPS)
    a, b, q = STEP
    for _ in range(c["steps"]):
        k = torch.mm(x.t(), x)
        p = torch.addmm(k, k, k, beta=b, alpha=q)
        p.diagonal().add_(a)
        x = torch.mm(x, p)
    x = x if tall else x.t()
    return s.alpha * x + (c["beta"] * s.C.double() if c["beta"] != 0.0 else 0.0)
