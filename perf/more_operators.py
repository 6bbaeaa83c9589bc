"""Cases that measure the operators between a linear layer's products and around its update.

With `own` false `run` computes an operator from elementary torch operations (the plain form);
with `own` true it makes the calls a user makes of the library's binding.

The operators and what a case of each stands for:
  qk_norm_rope           queries and keys as the QKV product leaves them -> every head normalised
                         (RMS over its values, times a weight) and rotated by its token's position
  qk_norm_rope_backward  gradients of the rotated heads -> gradients of the product's output (the
                         next data- and weight-gradient operand) and of both weights
  orthogonalize          a weight gradient or its momentum -> the update of the Muon optimiser: five
                         Newton-Schulz steps X <- a X + (b A + c A^2) X, A = X X^T, from G / |G|_F

Heads: q [T, Hq, D] and k [T, Hk, D] are views of one matrix [T, (Hq + 2 Hk) D], the product's
output (the values' heads are not touched).  The rotation turns `rotary` of a head's D values by
the angles of a table: row p holds cos and sin of p / base^(2 i / rotary), i < rotary / 2; the pairs are
(i, i + rotary / 2), or (2 i, 2 i + 1) interleaved.  A token with a negative position is padding:
its outputs and gradients are zeros.
"""
import math

import torch

own = False

EPS = 1e-6
STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
NORM_EPS = 1e-7


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # one token while decoding, far into a long context: latency
        dict(name="qk one token", op="qk_norm_rope", T=1, Hq=32, Hk=8, D=128, rotary=128,
             interleaved=False, dtype="bf16", head_major=False, table=131072, pad=0),
        # a ragged batch with padding: a product with FP32 output, heads of an odd size of which a part
        # is rotated
        dict(name="qk ragged", op="qk_norm_rope", T=333, Hq=40, Hk=10, D=80, rotary=32,
             interleaved=True, dtype="f32", head_major=True, table=4096, pad=21),
        # a training batch of the 8B-class layer (QKV 4096 -> 6144)
        dict(name="qk batch", op="qk_norm_rope", T=16384, Hq=32, Hk=8, D=128, rotary=128,
             interleaved=False, dtype="bf16", head_major=False, table=16384, pad=0),
        # the gradient of a small odd batch
        dict(name="qk backward ragged", op="qk_norm_rope_backward", T=257, Hq=16, Hk=4, D=64, rotary=64,
             interleaved=True, dtype="bf16", head_major=False, table=4096, pad=9),
        # wide heads, partly rotated, gradients laid out head by head, FP32 activations
        dict(name="qk backward wide", op="qk_norm_rope_backward", T=4096, Hq=16, Hk=4, D=256, rotary=64,
             interleaved=False, dtype="f32", head_major=True, table=8192, pad=0),
        # the gradient of the 8B-class layer's training batch
        dict(name="qk backward batch", op="qk_norm_rope_backward", T=16384, Hq=32, Hk=8, D=128,
             rotary=128, interleaved=False, dtype="bf16", head_major=False, table=16384, pad=0),
        # the weight of the smallest linear layer: a chain of small products
        dict(name="orthogonalize small", op="orthogonalize", E=1, R=512, C=512, dtype="f32"),
        # odd sizes, a gradient kept in bf16
        dict(name="orthogonalize odd", op="orthogonalize", E=1, R=1000, C=333, dtype="bf16"),
        # the keys' projection of the 8B-class layer: short and wide
        dict(name="orthogonalize wide", op="orthogonalize", E=1, R=1024, C=4096, dtype="f32"),
        # the weights of a layer of experts, each orthogonalised by itself
        dict(name="orthogonalize experts", op="orthogonalize", E=32, R=1408, C=2048, dtype="f32"),
        # a square projection
        dict(name="orthogonalize square", op="orthogonalize", E=1, R=4096, C=4096, dtype="f32"),
        # the 12B-class MLP's up-projection: tall, the largest
        dict(name="orthogonalize tall", op="orthogonalize", E=1, R=20480, C=5120, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "qk_norm_rope_backward", "orthogonalize"])
    if op == "orthogonalize":
        limit = work(listed()[-1])["flops"]
        while True:
            case = dict(op=op, E=rng.choice([1, 1, 1, _log_int(rng, 2, 32)]), R=_log_int(rng, 16, 20480),
                        C=_log_int(rng, 16, 8192), dtype=rng.choice(["bf16", "f32"]))
            if work(case)["flops"] <= limit and case["E"] * case["R"] * case["C"] <= 20480 * 5120:
                return case
    D = rng.choice([32, 64, 80, 96, 128, 192, 256])
    Hk = _log_int(rng, 1, 16)
    Hq = Hk * rng.choice([1, 2, 4, 5, 8])
    T = min(_log_int(rng, 1, 16384), 16384 * 5120 // ((Hq + Hk) * D))
    return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, rotary=rng.choice([D, D, 16 * rng.randint(1, D // 16)]),
                interleaved=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "f32"]),
                head_major=rng.random() < 0.4, table=_log_int(rng, 2048, 65536), pad=rng.choice([0, T // 9]))


# ---- inputs ----------------------------------------------------------------------------------

def _table(rows, rotary):
    i = torch.arange(rotary // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * i / rotary)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _positions(case, gen):
    """Packed sequences, each from its own start; the last `pad` tokens are padding."""
    T, rows = case["T"], case["table"]
    start = torch.rand(T, generator=gen, device="cuda") < 4.0 / T
    start[0] = True
    at = torch.arange(T, device="cuda")
    first = torch.cummax(torch.where(start, at, 0), 0).values
    base = torch.randint(0, rows, (T,), generator=gen, device="cuda")
    p = (base[first] + at - first) % rows
    if case["pad"]:
        p[T - case["pad"]:] = -1
    return p.int()


def _heads(T, H, D, head_major, dtype):
    """[T, H, D], stored by token or by head."""
    if head_major:
        return torch.zeros(H, T, D, dtype=dtype, device="cuda").transpose(0, 1)
    return torch.zeros(T, H, D, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["op"] == "orthogonalize":
        E, R, C = case["E"], case["R"], case["C"]
        g = 1e-3 * randn(E, R, C)
        spikes = torch.rand(E, R, C, generator=gen, device="cuda") < 0.005
        s["g"] = torch.where(spikes, 30.0 * g, g).to(dtype)
        s["out"] = torch.zeros(E, R, C, dtype=torch.bfloat16, device="cuda")
        return s
    T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
    qkv = randn(T, Hq + 2 * Hk, D)
    qkv *= torch.exp(0.5 * randn(1, Hq + 2 * Hk, 1))  # heads of different sizes
    qkv = qkv.to(dtype)
    s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    s["cos_sin"] = _table(case["table"], case["rotary"])
    s["positions"] = _positions(case, gen)
    s["q_weight"], s["k_weight"] = 1.0 + 0.1 * randn(D), 1.0 + 0.1 * randn(D)
    if case["op"] == "qk_norm_rope":
        s["q_out"] = _heads(T, Hq, D, case["head_major"], torch.bfloat16)
        s["k_out"] = _heads(T, Hk, D, case["head_major"], torch.bfloat16)
        return s
    for name, H in (("dq", Hq), ("dk", Hk)):
        d = _heads(T, H, D, case["head_major"], torch.bfloat16)
        d.copy_(1e-3 * randn(T, H, D))
        s[name] = d
    dqkv = torch.zeros(T, Hq + 2 * Hk, D, dtype=torch.bfloat16, device="cuda")
    s["dq_in"], s["dk_in"] = dqkv[:, :Hq], dqkv[:, Hq:Hq + Hk]
    return s


# ---- the framework's calls -------------------------------------------------------------------

def _run_own(s):
    from nvfp4_bit_quantized_03_b200 import binding as B
    if s["op"] == "orthogonalize":
        return B.orthogonalize(s["g"], steps=STEPS, coefficients=COEFFICIENTS, eps=NORM_EPS, out=s["out"])
    if s["op"] == "qk_norm_rope":
        return B.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["q_weight"], s["k_weight"],
                              eps=EPS, interleaved=s["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
    return B.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["cos_sin"],
                                   s["q_weight"], s["k_weight"], eps=EPS, interleaved=s["interleaved"],
                                   dq_in=s["dq_in"], dk_in=s["dk_in"])


# ---- the plain forms -------------------------------------------------------------------------

def _turn(x, cos, sin, interleaved):
    """The first 2 n values of every head turned by the angles with cosines cos [T, 1, n]."""
    n = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _angles(s):
    there = s["positions"] >= 0
    row = s["cos_sin"][s["positions"].clamp_min(0).long()][:, None]
    n = s["rotary"] // 2
    return row[..., :n], row[..., n:], there[:, None, None]


def _plain_qk(s):
    cos, sin, there = _angles(s)
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        out.append(torch.where(there, _turn(y, cos, sin, s["interleaved"]), 0.0).bfloat16())
    return tuple(out)


def _plain_qk_backward(s):
    cos, sin, there = _angles(s)
    grads, weights = [], []
    for x, w, d in ((s["q"], s["q_weight"], s["dq"]), (s["k"], s["k_weight"], s["dk"])):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        dy = torch.where(there, _turn(d.float(), cos, -sin, s["interleaved"]), 0.0)
        weights.append((dy * n).sum((0, 1), dtype=torch.float64).float())
        dn = dy * w
        grads.append((r * (dn - n * (dn * n).mean(-1, keepdim=True))).bfloat16())
    return tuple(grads + weights)


def _plain_orthogonalize(s):
    a, b, c = COEFFICIENTS
    x = s["g"].float()
    if s["R"] > s["C"]:
        x = x.transpose(1, 2)
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt() + NORM_EPS).float()
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if s["R"] > s["C"]:
        x = x.transpose(1, 2)
    return x.bfloat16().contiguous()


_PLAIN = dict(qk_norm_rope=_plain_qk, qk_norm_rope_backward=_plain_qk_backward,
              orthogonalize=_plain_orthogonalize)


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    if case["op"] == "orthogonalize":
        E, R, C = case["E"], case["R"], case["C"]
        m, n = min(R, C), max(R, C)
        # of the symmetric products (A and A^2) one half
        return {"bytes": E * R * C * ((2 if case["dtype"] == "bf16" else 4) + 2),
                "flops": STEPS * E * (3 * m * m * n + m * m * m)}
    T, D = case["T"], case["D"]
    real = T - case["pad"]
    heads = (case["Hq"] + case["Hk"]) * D
    size = 2 if case["dtype"] == "bf16" else 4
    table = 4 * case["rotary"] * min(real, case["table"])
    if case["op"] == "qk_norm_rope":
        return {"bytes": heads * (real * size + T * 2) + table + 4 * T + 8 * D, "flops": 10 * real * heads}
    return {"bytes": heads * (real * (size + 2) + T * 2) + table + 4 * T + 16 * D,
            "flops": 20 * real * heads}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _rotated(y, s):
    """Heads as complex numbers times exp(i angle); y [T, H, D] in FP64."""
    n = s["rotary"] // 2
    row = s["cos_sin"].double()[s["positions"].clamp_min(0).long()]
    phase = torch.complex(row[:, :n], row[:, n:])[:, None]
    if s["interleaved"]:
        z = torch.view_as_complex(y[..., :2 * n].unflatten(-1, (n, 2)).contiguous()) * phase
        front = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :n].contiguous(), y[..., n:2 * n].contiguous()) * phase
        front = torch.cat([z.real, z.imag], -1)
    out = torch.cat([front, y[..., 2 * n:]], -1)
    return out * (s["positions"] >= 0)[:, None, None]


def _normalised(x, w):
    return w * x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonalize":
        a, b, c = COEFFICIENTS
        out = []
        for g in s["g"]:
            x = g.double()
            x = x / (torch.linalg.vector_norm(x) + NORM_EPS)
            for _ in range(STEPS):
                if case["R"] > case["C"]:  # the Gram matrix of the columns, from the right
                    gram = x.T @ x
                    x = a * x + (b * x + c * (x @ gram)) @ gram
                else:
                    gram = x @ x.T
                    x = a * x + gram @ (b * x + c * (gram @ x))
            out.append(x)
        return torch.stack(out)
    heads = [(s["q"], s["q_weight"], s.get("dq")), (s["k"], s["k_weight"], s.get("dk"))]
    if case["op"] == "qk_norm_rope":
        return tuple(_rotated(_normalised(x.double(), w.double()), s) for x, w, _ in heads)
    dx, dw = [], []
    for x, w, d in heads:
        x, w = x.double().requires_grad_(), w.double().requires_grad_()
        gx, gw = torch.autograd.grad(_rotated(_normalised(x, w), s), (x, w), d.double())
        dx.append(gx)
        dw.append(gw)
    return tuple(dx + dw)
