"""Cases that measure the operators of a mixture-of-experts feed-forward layer in NVFP4.

With `own` false `run` computes an operator from elementary torch operations (the plain form);
with `own` true it makes the calls a user makes of the library's binding.

The operators and what a case of each stands for:
  route             router scores -> experts and weights of every token, and the plan of the
                    expert-ordered rows (tokens, one to a whole batch)
  route_backward    gradient of the weights -> gradient of the logits
  experts_fprop     tokens gathered into expert order, quantized (1x16 RTN), times W_e^T
  experts_dgrad     expert-ordered gradient, quantized stochastically, times W_e
  experts_wgrad     dW_e = dY_e^T X_e of Hadamard-transformed, quantized operands
  combine           weighted sum of each token's rows (or, without weights, their sum: the
                    backward pass of the gather)
  combine_backward  gradient of the rows and of the weights

Expert order: expert e owns the rows offsets[e] .. offsets[e + 1] of a matrix of `rows` rows, its
pairs (token, slot) first in the order of their index, then zero rows up to a multiple of 128.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
FLT_MAX = torch.finfo(torch.float32).max


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # one token while decoding: latency of the router and its plan
        dict(name="route one token", op="route", T=1, E=64, k=6, sigmoid=False, bias=False,
             groups=1, top_groups=1, scale=1.0, dtype="bf16", pad=0),
        # a training batch with many small experts, scores with a balancing bias, limited to groups
        dict(name="route batch", op="route", T=16384, E=256, k=8, sigmoid=True, bias=True,
             groups=8, top_groups=4, scale=2.5, dtype="f32", pad=100),
        # the router's gradient of a training batch
        dict(name="route backward", op="route_backward", T=8192, E=128, k=8, sigmoid=False,
             renorm=True, scale=1.0, dtype="bf16"),
        # one token through its experts while decoding: bound by the weights' bytes
        dict(name="fprop one token", op="experts_fprop", T=1, E=64, k=8, I=4096, O=4096, pad=0),
        # a ragged serving batch of odd size, part of it padding
        dict(name="fprop ragged", op="experts_fprop", T=257, E=32, k=4, I=2048, O=1408, pad=19),
        # a training batch, the up-projection of every expert
        dict(name="fprop batch", op="experts_fprop", T=8192, E=64, k=8, I=4096, O=2048, pad=0),
        # the data gradient of a mid-sized batch
        dict(name="dgrad", op="experts_dgrad", T=3000, E=16, k=2, I=5120, O=1536, pad=0),
        # the weight gradients: a small odd batch, and a training batch
        dict(name="wgrad ragged", op="experts_wgrad", T=333, E=8, k=2, I=1024, O=768, pad=13),
        dict(name="wgrad batch", op="experts_wgrad", T=8192, E=32, k=4, I=4096, O=2048, pad=0),
        # a few tokens while decoding
        dict(name="combine few", op="combine", T=16, E=64, k=8, C=4096, weighted=True, pad=0),
        # a training batch
        dict(name="combine batch", op="combine", T=8192, E=64, k=8, C=4096, weighted=True, pad=0),
        # its gradient
        dict(name="combine backward", op="combine_backward", T=4096, E=32, k=6, C=2048, pad=50),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "experts_fprop", "experts_fprop", "experts_dgrad",
                     "experts_wgrad", "combine", "combine_backward"])
    if op in ("route", "route_backward"):
        T = _log_int(rng, 1, 16000)
        sigmoid = rng.random() < 0.5
        dtype = rng.choice(["bf16", "f32"])
        scale = rng.choice([1.0, 2.5])
        if op == "route":
            groups = rng.choice([1, 1, 2, 4, 8])
            top = rng.randint(1, groups)
            E = groups * _log_int(rng, 4, 256 // groups)
            k = rng.randint(1, min(8, E // groups * top))
            return dict(op=op, T=T, E=E, k=k, sigmoid=sigmoid, bias=rng.random() < 0.5,
                        groups=groups, top_groups=top, scale=scale, dtype=dtype,
                        pad=rng.choice([0, T // 5]))
        E = _log_int(rng, 2, 256)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), sigmoid=sigmoid,
                    renorm=rng.random() < 0.5, scale=scale, dtype=dtype)
    E = _log_int(rng, 1, 64)
    k = rng.randint(1, min(8, E))
    if op in ("combine", "combine_backward"):
        T = _log_int(rng, 1, 8000)
        case = dict(op=op, T=T, E=E, k=k, C=8 * _log_int(rng, 8, 512), pad=rng.choice([0, T // 7]))
        if op == "combine":
            case["weighted"] = rng.random() < 0.5
        return case
    T = _log_int(rng, 1, 6000)
    E = min(E, 32)
    return dict(op=op, T=T, E=E, k=min(k, 4, E), I=64 * _log_int(rng, 2, 64),
                O=128 * _log_int(rng, 1, 16), pad=rng.choice([0, T // 7]))


# ---- inputs ----------------------------------------------------------------------------------

def _rows(T, E, k):
    """Rows of an expert-ordered matrix that hold every routing of T tokens."""
    pairs = T * k
    return (pairs + min(E, pairs) * 127) // 128 * 128


def _plan(experts, E, rows):
    """offsets [E + 1], pair_row [T, k] and row_token [rows] of a routing, in int32."""
    T, k = experts.shape
    dev = experts.device
    key = torch.where(experts >= 0, experts, E).reshape(-1).long()
    counts = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    counts.scatter_add_(0, key, torch.ones_like(key))
    first = counts.cumsum(0) - counts
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    offsets[1:] = ((counts[:E] + 127) // 128 * 128).cumsum(0)
    order = torch.argsort(key, stable=True)
    sorted_key = key[order]
    at = torch.arange(T * k, device=dev) - first[sorted_key] + offsets[sorted_key]
    at = torch.where(sorted_key < E, at, -1)
    pair_row = torch.empty(T * k, dtype=torch.int64, device=dev)
    pair_row[order] = at
    # one row more takes the pairs without an expert
    row_token = torch.full((rows + 1,), -1, dtype=torch.int64, device=dev)
    row_token[torch.where(at >= 0, at, rows)] = order // k
    return offsets.int(), pair_row.int().reshape(T, k), row_token[:rows].int()


def _routing(case, gen):
    """Experts of every token: distinct, some experts more popular; the last `pad` tokens none."""
    T, E, k = case["T"], case["E"], case["k"]
    popularity = 0.5 * torch.randn(E, generator=gen, device="cuda")
    noise = torch.rand(T, E, generator=gen, device="cuda").clamp_min(1e-7)
    experts = torch.topk(popularity - torch.log(-torch.log(noise)), k, dim=1).indices.int()
    if case.get("pad", 0):
        experts[T - case["pad"]:] = -1
    return experts


def _with_spikes(x, gen, frac, mult):
    return x * torch.where(torch.rand(x.shape, generator=gen, device="cuda") < frac, mult, 1.0)


def _swizzle(scales):
    """Row-major block scales [R, K / 16] -> the 128 x 4 tiles the tensor cores read, flat."""
    R, nb = scales.shape
    pad = -R % 128
    if pad:
        scales = torch.cat([scales, scales.new_zeros(pad, nb)])
    return scales.view(-1, 4, 32, nb // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _unswizzle(flat, R, nb):
    t = flat.view(-1, nb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(-1, nb)[:R]


def _weights(case, gen, transposed):
    """E weight matrices [O, I] stacked by rows, quantized with one scale per 16 x 16 block:
    the operand along I, or (transposed) the operand of the transpose along E * O."""
    E, I, O = case["E"], case["I"], case["O"]
    R = E * O
    codes = torch.empty(R, I // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(R, I // 16, dtype=torch.uint8, device="cuda")
    amax = torch.full((1,), 0.125, device="cuda")
    s_enc = _tensor_scale(amax)
    for r0 in range(0, R, 16384):
        n = min(16384, R - r0)
        w = (0.02 * torch.randn(n, I, generator=gen, device="cuda")).clamp(-0.125, 0.125)
        w = w.bfloat16().float()
        b = w.abs().view(n // 16, 16, I // 16, 16).amax(dim=(1, 3)).repeat_interleave(16, 0)
        sf = _scale_code(b, s_enc)
        r = _element_factor(sf.float(), s_enc).repeat_interleave(16, 1)
        index = _nearest(w.abs() * r)
        nib = (index + 8 * (w < 0)).to(torch.uint8).view(n, I // 2, 2)
        codes[r0:r0 + n] = nib[..., 0] | (nib[..., 1] << 4)
        scales[r0:r0 + n] = sf.view(torch.uint8)
    if transposed:
        nib = torch.stack([codes & 15, codes >> 4], -1).view(R, I).t()
        codes = (nib[:, 0::2] | (nib[:, 1::2] << 4)).contiguous()
        scales = scales.view(E * O // 16, 16, I // 16)[:, 0].t().repeat_interleave(16, 0)
    return codes, _swizzle(scales.contiguous()), amax


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case, seed=seed % (1 << 31))
    if op in ("route", "route_backward"):
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["logits"] = (1.5 * randn(T, E)).to(dtype)
        if op == "route":
            if case["pad"]:
                s["logits"][T - case["pad"]:] = -math.inf
            s["b"] = 0.1 * randn(E) if case["bias"] else None
        else:
            s["experts"] = _routing(case, gen)
            s["dweights"] = 1e-2 * randn(T, k)
        return s
    s["rows"] = rows = _rows(T, E, k)
    experts = _routing(case, gen)
    s["offsets"], s["pair_row"], s["row_token"] = _plan(experts, E, rows)
    s["total"] = total = int(s["offsets"][E])
    size = s["offsets"][1:] - s["offsets"][:-1]
    s["most"] = int(size.max())
    s["active"] = torch.nonzero(size > 0)[:, 0]  # the experts that have tokens
    valid = (s["row_token"] >= 0)[:, None]
    if op in ("combine", "combine_backward"):
        C = case["C"]
        y = torch.where(valid, randn(rows, C), 0.0)
        s["y"] = y.bfloat16()
        w = torch.rand(T, k, generator=gen, device="cuda") + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        if op == "combine":
            s["out"] = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
        else:
            s["dout"] = (1e-3 * randn(T, C)).bfloat16()
            s["dy"] = torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda")
        return s
    I, O = case["I"], case["O"]
    if op != "experts_dgrad":
        s["x"] = _with_spikes(randn(T, I), gen, 0.01, 50.0).bfloat16()
    if op != "experts_fprop":
        dy = torch.where(valid, _with_spikes(1e-3 * randn(rows, O), gen, 0.005, 100.0), 0.0)
        s["dy"] = dy.bfloat16()
        del dy
    if op == "experts_fprop":
        s["w"] = _weights(case, gen, False)
        s["out"] = torch.zeros(rows, O, dtype=torch.bfloat16, device="cuda")
    elif op == "experts_dgrad":
        s["w"] = _weights(case, gen, True)
        s["out"] = torch.zeros(rows, I, dtype=torch.bfloat16, device="cuda")
    else:
        s["sign_mask"] = int(torch.randint(0, 1 << 16, (1,), generator=gen, device="cuda"))
        s["out"] = torch.zeros(E * O, I, dtype=torch.float32, device="cuda")
    return s


# ---- the framework's calls -------------------------------------------------------------------

def _run_own(s):
    from nvfp4_bit_quantized_03_b200 import binding as B
    op = s["op"]
    if op == "route":
        experts, weights = B.route(s["logits"], s["k"], bias=s["b"], sigmoid=s["sigmoid"],
                                   groups=s["groups"], top_groups=s["top_groups"], renorm=True,
                                   scale=s["scale"])
        plan = B.expert_plan(experts, s["E"])
        return experts, weights, plan.offsets, plan.pair_row, plan.row_token
    if op == "route_backward":
        return B.route_backward(s["logits"], s["experts"], s["dweights"], sigmoid=s["sigmoid"],
                                renorm=s["renorm"], scale=s["scale"])
    plan = B.ExpertPlan(s["offsets"], s["pair_row"], s["row_token"])
    if op == "combine":
        return B.combine(s["y"], plan, s["weights"] if s["weighted"] else None, out=s["out"])
    if op == "combine_backward":
        return B.combine_backward(s["dout"], s["y"], plan, s["weights"], dy=s["dy"])
    if op == "experts_wgrad":
        return B.experts_wgrad(s["dy"], s["x"], plan, s["sign_mask"], s["seed"], 0, out=s["out"])
    w = B.QuantizedTensor.from_buffers(*s["w"])
    if op == "experts_fprop":
        return B.experts_fprop(s["x"], w, plan, out=s["out"])
    return B.experts_dgrad(s["dy"], w, plan, s["seed"], 0, out=s["out"])


# ---- the plain forms -------------------------------------------------------------------------

def _over(a, b):
    """a / b rounded to nearest: torch divides two tensors, but takes the quotient of a tensor and
    a number as a product with a rounded reciprocal."""
    return torch.as_tensor(a, dtype=b.dtype, device=b.device).expand_as(b) / b


def _tensor_scale(amax):
    return torch.where(amax == 0, 1.0, _over(2688.0, amax).clamp(max=FLT_MAX))


def _scale_code(b, s_enc):
    """E4M3 code of (b / 6) s_enc."""
    return ((b / torch.full_like(b, 6.0)) * s_enc).clamp(max=448).to(torch.float8_e4m3fn)


def _element_factor(sf, s_enc):
    return torch.where(sf > 0, (s_enc / sf.clamp_min(2.0 ** -9)).clamp(max=FLT_MAX), 0.0)


def _nearest(v):
    """E2M1 magnitude code nearest to v >= 0, ties to the even code."""
    return ((v > 0.25).byte() + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5)
            + (v > 5.0))


def _philox(groups, seed, offset):
    """Philox-4x32-10 of counters (group, offset) under the key `seed`: [n, 8] 16-bit values."""
    low = 0xFFFFFFFF
    c0, c1 = groups & low, groups >> 32
    c2 = torch.full_like(groups, offset & low)
    c3 = torch.full_like(groups, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], -1)
    return torch.stack([words & 0xFFFF, words >> 16], -1).reshape(-1, 8)


def _stochastic(v, random16):
    """E2M1 magnitude code of v >= 0, rounded up where random16 < 65536 (v - lo) / (hi - lo)."""
    grid = torch.tensor(GRID, device=v.device)
    low = ((v >= 0.5).byte() + (v >= 1.0) + (v >= 1.5) + (v >= 2.0) + (v >= 3.0) + (v >= 4.0)
           + (v >= 6.0)).int()
    lo, hi = grid[low], grid[(low + 1).clamp(max=7)]
    p = torch.where(low < 7, (v - lo) / (hi - lo).clamp_min(0.5), 0.0)
    return low + (random16 < p * 65536.0)


def _quantized(y, amax, seed=None, offset=0):
    """Rows of y (FP32) quantized in blocks of 16: (code value x block scale, tensor scale).
    With a seed the rounding is stochastic, element (r, c) drawing lane r * cols + c."""
    R, C = y.shape
    s_enc = _tensor_scale(amax)
    b = y.abs().view(R, C // 16, 16).amax(-1)
    sf = _scale_code(b, s_enc).float()
    v = y.abs() * _element_factor(sf, s_enc).repeat_interleave(16, 1)
    if seed is None:
        index = _nearest(v)
    else:
        groups = torch.arange(R * C // 8, device=y.device)
        index = _stochastic(v, _philox(groups, seed, offset).view(R, C))
    value = torch.tensor(GRID, device=y.device)[index.int()] * torch.sign(y)
    return value * sf.repeat_interleave(16, 1), s_enc


def _hadamard16(x, sign_mask):
    """(1/4) H diag(s) over every 16 consecutive values of the last axis, FP32 butterflies."""
    R, C = x.shape
    sign = torch.tensor([-1.0 if sign_mask >> i & 1 else 1.0 for i in range(16)], device=x.device)
    v = (x.view(R, C // 16, 16) * sign).view(-1, 16)
    for width in (1, 2, 4, 8):
        v = v.view(-1, 16 // (2 * width), 2, width)
        v = torch.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2).view(-1, 16)
    return (0.25 * v).view(R, C)


def _stored(operand, rows, cols):
    """(code value x block scale, tensor scale) of a stored operand."""
    codes, scales, amax = operand
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([grid[byte & 15], grid[byte >> 4]], -1)
    value = pairs[codes.int()].view(rows, cols // 16, 16)
    sf = _unswizzle(scales, rows, cols // 16).contiguous().view(torch.float8_e4m3fn).float()
    return (value * sf[..., None]).view(rows, cols), _tensor_scale(amax)


def _regions(s, experts):
    """[experts, most] rows of these experts' regions (clamped), and which of them are inside."""
    start, end = s["offsets"][experts].long(), s["offsets"][experts + 1].long()
    at = start[:, None] + torch.arange(max(1, s["most"]), device=start.device)
    return at.clamp(max=s["rows"] - 1), at < end[:, None]


def _gathered(s):
    """Tokens in expert order (FP32), zeros in the rows without a token."""
    token = s["row_token"]
    return torch.where(token[:, None] >= 0, s["x"].float()[token.clamp_min(0).long()], 0.0)


def _product(s, a, w):
    """The active experts' rows of a [rows, K] times their w [active, N, K]^T: [total, N], FP32."""
    at, inside = _regions(s, s["active"])
    blocks = torch.where(inside[..., None], a[at], 0.0)
    row = torch.arange(s["total"], device=a.device)
    e = torch.searchsorted(s["offsets"][s["active"] + 1].long(), row, right=True)
    slot = e * max(1, s["most"]) + row - s["offsets"][s["active"]].long()[e]
    return torch.bmm(blocks, w.transpose(1, 2)).view(-1, w.shape[1])[slot]


def _plain_fprop(s):
    E, I, O, total = s["E"], s["I"], s["O"], s["total"]
    x = _gathered(s)
    a, sa = _quantized(x, x.abs().amax())
    codes, scales, amax = s["w"]
    n = s["active"].numel()  # an expert's codes and scales are contiguous
    w, sw = _stored((codes.view(E, -1)[s["active"]], scales.view(E, -1)[s["active"]], amax), n * O, I)
    y = torch.zeros(s["rows"], O, dtype=torch.bfloat16, device=x.device)
    y[:total] = (_product(s, a, w.view(n, O, I)) * (1.0 / (sa.double() * sw)).float()).bfloat16()
    return y


def _plain_dgrad(s):
    E, I, O, total = s["E"], s["I"], s["O"], s["total"]
    dy = s["dy"].float()
    a, sa = _quantized(dy, dy.abs().amax(), s["seed"], 0)
    codes, scales, amax = s["w"]
    n = s["active"].numel()  # an expert's columns of the codes, its column tiles of the scales
    codes = codes.view(I, E, O // 2)[:, s["active"]].reshape(I, -1)
    scales = scales.view(-1, E, O // 64, 512)[:, s["active"]].reshape(-1)
    w, sw = _stored((codes, scales, amax), I, n * O)
    dx = torch.zeros(s["rows"], I, dtype=torch.bfloat16, device=dy.device)
    d = _product(s, a, w.view(I, n, O).transpose(0, 1))
    dx[:total] = (d * (1.0 / (sa.double() * sw)).float()).bfloat16()
    return dx


def _plain_wgrad(s):
    at, inside = _regions(s, torch.arange(s["E"], device=s["dy"].device))

    def operand(x, seed, offset):
        t = _hadamard16(x.t().contiguous(), s["sign_mask"])
        q, scale = _quantized(t, t.abs().amax(), seed, offset)
        return torch.where(inside, q[:, at], 0.0).transpose(0, 1), scale

    a, sa = operand(s["dy"].float(), s["seed"], 1)
    b, sb = operand(_gathered(s), None, 0)
    d = torch.bmm(a, b.transpose(1, 2)) * (1.0 / (sa.double() * sb)).float()
    return d.reshape(s["E"] * s["O"], s["I"])


def _plain_route(s):
    logits, k, E, groups = s["logits"].double(), s["k"], s["E"], s["groups"]
    T = logits.shape[0]
    open_ = logits > -math.inf
    if s["sigmoid"]:
        log_score = torch.nn.functional.logsigmoid(logits)
    else:
        log_score = logits - logits.amax(1, keepdim=True).clamp_min(-1e300)
        log_score = log_score - torch.log(log_score.exp().sum(1, keepdim=True))
    log_score = torch.where(open_, log_score, -math.inf)
    if s["b"] is None and groups == 1:
        choice = logits
    else:
        choice = log_score.exp() + (0.0 if s["b"] is None else s["b"].double())
        choice = torch.where(open_, choice, -math.inf)
    if groups > 1:
        best = torch.sort(choice.view(T, groups, E // groups), dim=2, descending=True).values[..., :2]
        score = torch.where(best > -math.inf, best, 0.0).sum(2)
        score = torch.where(best[..., 0] > -math.inf, score, -math.inf)
        keep = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        kept = torch.zeros(T, groups, dtype=torch.bool, device=logits.device).scatter_(1, keep, True)
        choice = torch.where(kept.repeat_interleave(E // groups, 1), choice, -math.inf)
    value, index = torch.sort(choice, dim=1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k]
    chosen = value > -math.inf
    picked = torch.where(chosen, log_score.gather(1, index), -math.inf)
    picked = picked - picked[:, :].amax(1, keepdim=True).clamp_min(-1e300)
    share = picked.exp()
    share = torch.where(chosen, share / share.sum(1, keepdim=True).clamp_min(1e-300), 0.0)
    experts = torch.where(chosen, index, -1).int()
    weights = (share * s["scale"]).float()
    return (experts, weights) + _plan(experts, E, _rows(T, E, k))


def _plain_route_backward(s):
    logits, scale = s["logits"].float(), s["scale"]
    index = s["experts"].long()
    chosen = torch.where(index >= 0, 1.0, 0.0)
    index = index.clamp_min(0)
    dw = s["dweights"] * chosen * scale
    if s["sigmoid"]:
        score = torch.sigmoid(logits)
        local = 1.0 - score
    else:
        score = torch.softmax(logits, 1)
        local = torch.ones_like(score)
    picked = score.gather(1, index) * chosen
    dlogits = torch.zeros_like(logits)
    if s["renorm"]:
        share = picked / picked.sum(1, keepdim=True).clamp_min(1e-30)
        g = share * (dw - (dw * share).sum(1, keepdim=True)) * local.gather(1, index)
    else:
        g = picked * dw * local.gather(1, index)
        if not s["sigmoid"]:
            dlogits = dlogits - score * (dw * picked).sum(1, keepdim=True)
    return dlogits.scatter_add(1, index, g).to(s["logits"].dtype)


def _plain_combine(s):
    row = s["pair_row"].long()
    weight = torch.where(row >= 0, s["weights"] if s["weighted"] else 1.0, 0.0)
    return (s["y"][row.clamp_min(0)].float() * weight[..., None]).sum(1).bfloat16()


def _plain_combine_backward(s):
    row = s["pair_row"].long()
    there = row >= 0
    dout = s["dout"].float()
    y = s["y"][row.clamp_min(0)].float()
    dweights = torch.where(there, (y * dout[:, None]).sum(2), 0.0)
    # one row more takes the pairs without an expert
    dy = torch.zeros(s["rows"] + 1, s["C"], dtype=torch.bfloat16, device=dout.device)
    dy[torch.where(there, row, s["rows"])] = (dout[:, None] * s["weights"][..., None]).bfloat16()
    return dy[:s["rows"]], dweights


_PLAIN = dict(route=_plain_route, route_backward=_plain_route_backward, combine=_plain_combine,
              combine_backward=_plain_combine_backward, experts_fprop=_plain_fprop,
              experts_dgrad=_plain_dgrad, experts_wgrad=_plain_wgrad)


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    P = (T - case.get("pad", 0)) * k
    if op in ("route", "route_backward"):
        size = 2 if case["dtype"] == "bf16" else 4
        if op == "route":
            return {"bytes": T * E * size + T * k * 12 + 4 * _rows(T, E, k), "flops": 8 * T * E}
        return {"bytes": 2 * T * E * size + T * k * 8, "flops": 8 * T * E}
    if op == "combine":
        C = case["C"]
        return {"bytes": 2 * C * (P + T) + T * k * (8 if case["weighted"] else 4),
                "flops": 2 * P * C}
    if op == "combine_backward":
        C = case["C"]
        return {"bytes": 2 * C * (2 * P + T) + T * k * 12, "flops": 3 * P * C}
    I, O = case["I"], case["O"]
    active = E * (1 - (1 - k / E) ** (T - case["pad"]))
    flops = 2 * P * I * O
    if op == "experts_fprop":
        return {"bytes": (T - case["pad"]) * I * 2 + active * I * O * 9 / 16 + P * O * 2, "flops": flops}
    if op == "experts_dgrad":
        return {"bytes": P * O * 2 + active * I * O * 9 / 16 + P * I * 2, "flops": flops}
    return {"bytes": P * O * 2 + (T - case["pad"]) * I * 2 + E * I * O * 4, "flops": flops}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _exact_blocks(y, amax, seed=None, offset=0):
    """Dequantized rows of y (FP64 holding FP32 values).  The definition fixes FP32 roundings for
    the scales and the scaled elements; they are taken in FP64 and rounded, which gives the same
    bits as one FP32 operation."""
    def f32(t):
        return t.float().double()

    R, C = y.shape
    scale = f32(2688.0 / amax) if float(amax) else torch.ones_like(amax)
    block = y.reshape(R, C // 16, 16)
    t = f32(f32(block.abs().amax(2) / 6.0) * scale).clamp(max=448.0)
    exponent = torch.frexp(t).exponent.clamp(min=-5).double() - 1
    quantum = torch.exp2(exponent - 3)
    sf = torch.round(t / quantum) * quantum
    factor = torch.where(sf > 0, f32(scale / torch.where(sf > 0, sf, 1.0)), 0.0)
    v = f32(block.abs() * factor[..., None]).reshape(R, C)
    grid = torch.tensor(GRID, dtype=torch.float64, device=y.device)
    above = torch.searchsorted(grid, v, right=True).clamp(max=7)
    lo, hi = grid[above - 1], grid[above]
    if seed is None:
        middle = (lo + hi) / 2
        up = (v > middle) | ((v == middle) & (above % 2 == 0))
    else:
        draw16 = _philox(torch.arange(R * C // 8, device=y.device), seed, offset).view(R, C)
        up = draw16 < (v - lo) / (hi - lo) * 65536
    value = torch.where(up, hi, lo) * torch.sign(y)
    return (value.view(R, C // 16, 16) * (sf / scale)[..., None]).view(R, C)


def _exact_weights(operand, rows, cols):
    codes, scales, amax = operand
    nibble = torch.stack([codes & 15, codes >> 4], 2).view(rows, cols)
    grid = torch.tensor(GRID, dtype=torch.float64, device=codes.device)
    value = grid[(nibble & 7).int()] * torch.where(nibble > 7, -1.0, 1.0)
    r = torch.arange(rows, device=codes.device)[:, None]
    j = torch.arange(cols // 16, device=codes.device)[None]
    place = ((r // 128) * (cols // 64) + j // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + j % 4
    sf = scales[place].view(torch.float8_e4m3fn).double()
    return value * sf.repeat_interleave(16, 1) / (2688.0 / amax).float().double()


def exact(case, seed):
    op = case["op"]
    if op.startswith("experts") and work(case)["flops"] > 1.2e11:
        return None
    s = prepare(case, seed)
    if op == "route":
        picked = _plain_route(dict(s, scale=1.0))[0].long()
        l = s["logits"].double()
        e = torch.sigmoid(l) if s["sigmoid"] else torch.exp(l - l.amax(1, keepdim=True))
        e = torch.where(picked >= 0, e.gather(1, picked.clamp_min(0)), 0.0)
        total = e.sum(1, keepdim=True)
        return None, torch.where(total > 0, s["scale"] * e / total, 0.0), None, None, None
    if op == "route_backward":
        l = s["logits"].double().requires_grad_()
        score = torch.sigmoid(l) if s["sigmoid"] else torch.softmax(l, 1)
        w = score.gather(1, s["experts"].long())
        w = s["scale"] * (w / w.sum(1, keepdim=True) if s["renorm"] else w)
        return torch.autograd.grad((w * s["dweights"].double()).sum(), l)[0]
    row = s["pair_row"].long()
    if op == "combine":
        out = torch.zeros(s["T"], s["C"], dtype=torch.float64, device="cuda")
        for j in range(s["k"]):
            w = torch.where(row[:, j] >= 0, s["weights"][:, j].double() if s["weighted"] else 1.0, 0.0)
            out += w[:, None] * s["y"][row[:, j].clamp_min(0)].double()
        return out
    if op == "combine_backward":
        y = s["y"].double().requires_grad_()
        w = s["weights"].double().requires_grad_()
        kept = torch.where(row >= 0, w, 0.0)
        out = (y[row.clamp_min(0)] * kept[..., None]).sum(1)
        return torch.autograd.grad((out * s["dout"].double()).sum(), (y, w))
    E, I, O, total = s["E"], s["I"], s["O"], s["total"]
    bounds = s["offsets"].tolist()
    x = None
    if "x" in s:
        x = s["x"].double()[s["row_token"].clamp_min(0).long()] * (s["row_token"] >= 0)[:, None]
    if op == "experts_wgrad":
        h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
        for _ in range(4):
            h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
        h = h / 4 * torch.tensor([-1.0 if s["sign_mask"] >> i & 1 else 1.0 for i in range(16)],
                                 dtype=torch.float64, device="cuda")
        def along_rows(m, *stream):
            t = (m.t().reshape(m.shape[1], -1, 16) @ h.t()).reshape(m.shape[1], -1).float().double()
            return _exact_blocks(t, t.abs().amax(), *stream)
        a, b = along_rows(s["dy"].double(), s["seed"], 1), along_rows(x)
        return torch.cat([a[:, p:q] @ b[:, p:q].t() for p, q in zip(bounds, bounds[1:])])
    if op == "experts_fprop":
        a, w = _exact_blocks(x, x.abs().amax()), _exact_weights(s["w"], E * O, I).view(E, O, I)
    else:
        dy = s["dy"].double()
        a = _exact_blocks(dy, dy.abs().amax(), s["seed"], 0)
        w = _exact_weights(s["w"], I, E * O).view(I, E, O).transpose(0, 1)
    out = torch.zeros(s["rows"], w.shape[1], dtype=torch.float64, device="cuda")
    out[:total] = torch.cat([a[p:q] @ w[e].t() for e, (p, q) in enumerate(zip(bounds, bounds[1:]))])
    return out
