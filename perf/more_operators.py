"""Cases, plain forms and calls of RMS norm with a residual, the gated feed-forward block, gradient clipping and the
relative position bias.

The operators as formulas (x a row of C channels; sums over the row unless said otherwise):

- RMS norm: r = x + residual, rounded to the type (x itself without a residual), rstd = 1 / sqrt(sum(r^2) / C + eps),
  y = r rstd gamma; also in 8 bits, y8: for every 128 consecutive channels of a row (the last group may be shorter)
  s = FP32(max|y| / 127), q = round-half-even(FP32(y FP32(127 / max|y|))), which stands for q s (zeros below 2^-120).
  Backward, with g = dy gamma and dr the gradient that reaches r from elsewhere:
  dx = rstd (g - r rstd^2 sum(g r) / C) + dr, dgamma = sum over rows of dy r rstd.
- Gated feed-forward block: a = x Wg^T, u = x Wu^T, h = act(a) u, out = h Wd^T (Wg, Wu [F, C], Wd [C, F]; act is
  a sigmoid(a), a Phi(a) or sigmoid(a)). Backward, from the a and u that the forward kept: dh = dout Wd,
  da = dh u act'(a), du = dh act(a), dx = da Wg + du Wu, dWg = da^T x, dWu = du^T x, dWd = dout^T h.
- Clipping: norm = sqrt(sum of all elements' squares), every gradient times min(1, most / (norm + 1e-6)).
- Relative position bias: n = |key's position - query's|, bucket k holds starts[k] <= n < starts[k + 1] (the last one all
  that are further away); with two sides the keys behind the query have buckets K + k, with one side they have n = 0.
  bias[b, h, i, j] = base[b, h, i, j] + table[bucket(i, j), h]; backward: dtable[t, h] = sum of dbias where bucket = t.
"""
import math

import torch

own = False

EPS = 1e-5
GROUP = 128
TINY = 2.0 ** -120
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MOST_VALUES = 768 * 768 * 128
MOST_FLOPS = 6 * 8192 * 4096 * 16384
MOST_GRADS = 400_000_000


def listed():
    return [
        # the single representation of a 384-residue crop with its residual: latency
        {"name": "rms_fwd_single", "op": "rms_fwd", "M": 384, "C": 384, "dtype": "bf16", "residual": True, "bits8": False},
        # a pre-norm layer's wide rows: the residual's sum, the normalised rows in 8 bits for the backward pass, brought back
        {"name": "rms_fwd_wide_8bit", "op": "rms_fwd", "M": 8192, "C": 4096, "dtype": "bf16", "residual": True, "bits8": True},
        # an odd width and an odd number of rows, with the gradient that comes past the layer
        {"name": "rms_bwd_odd", "op": "rms_bwd", "M": 20011, "C": 1003, "dtype": "fp16", "residual": True},
        # eight sequences' new tokens through a wide block: serving, bound by the weights
        {"name": "ffn_fwd_token", "op": "ffn_fwd", "M": 8, "C": 4096, "F": 16384, "act": "silu", "keep": False},
        # the transition of the pair representation at crop 384 (four times its channels)
        {"name": "ffn_fwd_pair384", "op": "ffn_fwd", "M": 147456, "C": 128, "F": 512, "act": "silu", "keep": False},
        # a long prompt through a wide block
        {"name": "ffn_fwd_long", "op": "ffn_fwd", "M": 8192, "C": 4096, "F": 16384, "act": "silu", "keep": False},
        # a training step's backward pass
        {"name": "ffn_bwd_long", "op": "ffn_bwd", "M": 8192, "C": 2048, "F": 8192, "act": "silu"},
        # ragged rows and widths that fill no tile, the other activation
        {"name": "ffn_bwd_odd", "op": "ffn_bwd", "M": 4001, "C": 392, "F": 1032, "act": "gelu"},
        # the gradients of eight triangle-attention blocks of 128 channels: many small tensors
        {"name": "clip_blocks", "op": "clip", "n": 40, "total": 661504, "dtype": "fp32", "clips": True},
        # a large model's gradients, of two types
        {"name": "clip_large", "op": "clip", "n": 50, "total": 300_000_007, "dtype": "mixed", "clips": True},
        # the pair bias of sixteen heads at the longest triangle axis, logarithmic buckets on top of the projected bias
        {"name": "relpos_fwd_1024", "op": "relpos_fwd", "B": 2, "H": 16, "Nq": 1024, "Nk": 1024, "K": 16, "far": 128, "two": True,
         "base": True, "chains": False},
        # its gradient at an odd length, with the positions of several chains
        {"name": "relpos_bwd_chains", "op": "relpos_bwd", "B": 2, "H": 16, "Nq": 1003, "Nk": 1003, "K": 33, "far": 33, "two": True,
         "base": True, "chains": True},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "ffn_fwd", "ffn_fwd", "ffn_bwd", "ffn_bwd", "clip", "relpos_fwd", "relpos_bwd"])
    if op in ("rms_fwd", "rms_bwd"):
        while True:
            M, C = _log_int(rng, 1, 600000), _log_int(rng, 8, 8192)
            if rng.random() < 0.6:
                C = (C + 7) // 8 * 8
            if 2000 <= M * C <= MOST_VALUES:
                case = {"op": op, "M": M, "C": C, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "residual": rng.random() < 0.7}
                return case if op == "rms_bwd" else {**case, "bits8": rng.random() < 0.5}
    if op in ("ffn_fwd", "ffn_bwd"):
        while True:
            M, C, F = _log_int(rng, 1, 150000), 8 * _log_int(rng, 8, 1024), 8 * _log_int(rng, 8, 2048)
            flops, values = (6 if op == "ffn_fwd" else 12) * M * C * F, M * (C + 3 * F)
            if 1e6 <= flops <= MOST_FLOPS and values <= 1_000_000_000 and C * F <= 4096 * 16384:
                case = {"op": op, "M": M, "C": C, "F": F, "act": rng.choice(["silu", "silu", "gelu", "sigmoid"])}
                return case if op == "ffn_bwd" else {**case, "keep": rng.random() < 0.4}
    if op == "clip":
        n = _log_int(rng, 1, 60)
        return {"op": op, "n": n, "total": max(n, _log_int(rng, 100, MOST_GRADS)), "dtype": rng.choice(["fp32", "bf16", "fp16", "mixed"]),
                "clips": rng.random() < 0.7}
    while True:
        B, H, Nq, Nk = rng.choice([1, 1, 2, 3, 4]), _log_int(rng, 1, 32), _log_int(rng, 1, 2048), _log_int(rng, 1, 2048)
        if rng.random() < 0.5:
            Nk = Nq
        if 2000 <= B * H * Nq * Nk <= 34_000_000:
            K = _log_int(rng, 2, 64)
            return {"op": op, "B": B, "H": H, "Nq": Nq, "Nk": Nk, "K": K, "far": rng.choice([K, 2 * K, 8 * K]), "two": rng.random() < 0.7,
                    "base": rng.random() < 0.5, "chains": rng.random() < 0.5}


def _sizes(case):
    """The tensors' sizes: weights that halve from one to the next, over and over, the first one with what is left."""
    n, total = case["n"], case["total"]
    shares = [2.0 ** -(i % 5) for i in range(n)]
    sizes = [max(1, int((total - n) * s / sum(shares))) for s in shares]
    sizes[0] += total - sum(sizes)
    return sizes


def _types(case):
    names = {"mixed": ["fp32", "bf16"]}.get(case["dtype"], [case["dtype"]])
    return [DTYPES[names[i % len(names)]] for i in range(case["n"])]


def work(case):
    op = case["op"]
    if op.startswith("rms"):
        M, C = case["M"], case["C"]
        x, q = M * C * DTYPES[case["dtype"]].itemsize, M * C + 4 * M * ((C + GROUP - 1) // GROUP)
        if op == "rms_bwd":  # r, dy (and dr) read, dx written
            return {"bytes": (4 if case["residual"] else 3) * x + 4 * M + 8 * C, "flops": 9 * M * C}
        move = (3 if case["residual"] else 1) * x + 4 * M + 4 * C
        if case["bits8"]:  # put away, brought back
            return {"bytes": move + 2 * q + x, "flops": 9 * M * C}
        return {"bytes": move + x, "flops": 5 * M * C}
    if op.startswith("ffn"):
        M, C, F = case["M"], case["C"], case["F"]
        if op == "ffn_fwd":
            return {"bytes": 2 * (2 * M * C + 3 * C * F + (2 * M * F if case["keep"] else 0)), "flops": 6 * M * C * F}
        return {"bytes": 2 * (3 * M * C + 6 * C * F + 2 * M * F), "flops": 12 * M * C * F}
    if op == "clip":
        size = sum(n * t.itemsize for n, t in zip(_sizes(case), _types(case)))
        return {"bytes": 2 * size + 4, "flops": 3 * case["total"]}
    values = case["B"] * case["H"] * case["Nq"] * case["Nk"]
    table = 4 * (2 if case["two"] else 1) * case["K"] * case["H"]
    if op == "relpos_fwd":
        return {"bytes": (4 if case["base"] else 2) * values + table, "flops": values}
    return {"bytes": 2 * values + table, "flops": values}


# ------------------------------------------------------------------------------------------------ inputs

def _starts(case):
    """The buckets' first distances, from whole numbers: one distance a bucket for the first half, the rest in equal
    steps of the logarithm up to `far` (bucket e + k from the smallest n on with (n / e)^m >= (far / e)^k, where
    m = K - e). All of them one distance each where far is K."""
    K, far = case["K"], case["far"]
    if far <= K:
        return list(range(K))
    e = (K + 1) // 2
    m, starts = K - e, list(range(e + 1))
    for k in range(1, m):
        n = starts[-1] + 1
        while n ** m * e ** k < far ** k * e ** m:
            n += 1
        starts.append(n)
    return starts[:K]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        x = torch.randn(shape, generator=gen, device="cuda")
        return x.mul_(std).add_(mean).to(dtype)

    op = case["op"]
    st = {"op": op}
    if op.startswith("rms"):
        M, C, dtype = case["M"], case["C"], DTYPES[case["dtype"]]
        st["x"] = normal(M, C, dtype=dtype, std=1.5, mean=0.1)
        st["gamma"] = normal(C, std=0.2, mean=1.0)
        if op == "rms_fwd":
            st["residual"] = normal(M, C, dtype=dtype, std=2.0) if case["residual"] else None
            st["bits8"] = case["bits8"]
        else:
            _, st["rstd"], _ = _rms_fwd(st["x"], st["gamma"], None)
            st["dy"] = normal(M, C, dtype=dtype)
            st["dr"] = normal(M, C, dtype=dtype) if case["residual"] else None
        return st
    if op.startswith("ffn"):
        M, C, F, bf = case["M"], case["C"], case["F"], torch.bfloat16
        st["act"] = case["act"]
        st["x"] = normal(M, C, dtype=bf)
        st["wg"], st["wu"] = normal(F, C, dtype=bf, std=C ** -0.5), normal(F, C, dtype=bf, std=C ** -0.5)
        st["wd"] = normal(C, F, dtype=bf, std=F ** -0.5)
        if op == "ffn_fwd":
            st["keep"] = case["keep"]
        else:  # (what the forward kept, and the gradient of its result)
            st["a"], st["u"] = (torch.matmul(st["x"], w.T) for w in (st["wg"], st["wu"]))
            st["dout"] = normal(M, C, dtype=bf)
        return st
    if op == "clip":
        sizes, types = _sizes(case), _types(case)
        st["grads"] = [normal(n, dtype=t, std=0.01 * (1 + i % 3)) for i, (n, t) in enumerate(zip(sizes, types))]
        st["out"] = [torch.empty_like(g) for g in st["grads"]]
        size = math.sqrt(sum(n * (0.01 * (1 + i % 3)) ** 2 for i, n in enumerate(sizes)))
        st["most"] = (0.25 if case["clips"] else 4.0) * size
        return st
    B, H, Nq, Nk = (case[k] for k in ("B", "H", "Nq", "Nk"))
    st["starts"], st["two"] = _starts(case), case["two"]
    st["Nq"], st["Nk"] = Nq, Nk
    st["table"] = normal((2 if case["two"] else 1) * case["K"], H)
    st["posq"] = st["posk"] = None
    if case["chains"]:  # several chains, numbered on with a gap between them, and residues missing here and there
        def places(n):
            steps = 1 + (torch.rand((B, n), generator=gen, device="cuda") < 0.05).int() + 200 * (
                torch.rand((B, n), generator=gen, device="cuda") < 3.0 / n).int()
            return torch.cumsum(steps, 1).int()

        st["posq"] = places(Nq)
        st["posk"] = st["posq"] if Nq == Nk else places(Nk)
    if op == "relpos_fwd":
        st["B"] = B
        st["base"] = normal(B, H, Nq, Nk, dtype=torch.bfloat16) if case["base"] else None
    else:
        st["dbias"] = normal(B, H, Nq, Nk, dtype=torch.bfloat16, std=0.1)
    return st


# ------------------------------------------------------------------------------------------------ plain forms

def _rms_fwd(x, gamma, residual):
    r = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    rf = r.float()
    rstd = 1.0 / torch.sqrt((rf * rf).mean(1) + EPS)
    return rf * rstd[:, None] * gamma, rstd, r


def _eight_bits(y):
    """What y [M, C] (in 32 bits) kept in 8 bits stands for."""
    M, C = y.shape
    n = (C + GROUP - 1) // GROUP
    g = torch.nn.functional.pad(y, (0, n * GROUP - C)).view(M, n, GROUP)
    top = g.abs().amax(2, keepdim=True)
    kept = top >= TINY
    most = torch.full_like(top, 127.0)  # a tensor: a quotient with a Python number goes by its rounded inverse
    s = torch.where(kept, top / most, torch.zeros_like(top))
    inv = torch.where(kept, most / top, torch.zeros_like(top))
    return (torch.round(g * inv).clamp(-127, 127) * s).view(M, n * GROUP)[:, :C]


def _rms_bwd(st):
    r, rstd, dy = st["x"].float(), st["rstd"][:, None], st["dy"].float()
    rh = r * rstd
    g = dy * st["gamma"]
    dx = rstd * (g - rh * (g * rh).mean(1, keepdim=True))
    if st["dr"] is not None:
        dx = dx + st["dr"].float()
    return dx.to(st["dy"].dtype), (dy * rh).sum(0)


def _act(a, act):
    """act(a) and its derivative."""
    if act == "gelu":
        phi = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
        return a * phi, phi + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2.0 * math.pi))
    s = 1.0 / (1.0 + torch.exp(-a))
    if act == "sigmoid":
        return s, s * (1.0 - s)
    return a * s, s * (1.0 + a * (1.0 - s))


def _ffn_fwd(st):
    x, bf = st["x"].float(), torch.bfloat16
    a, u = torch.matmul(x, st["wg"].float().T), torch.matmul(x, st["wu"].float().T)
    out = torch.matmul(_act(a, st["act"])[0] * u, st["wd"].float().T).to(bf)
    return (out, a.to(bf), u.to(bf)) if st["keep"] else out


def _ffn_bwd(st):
    x, wg, wu, wd, a, u, dout = (st[k].float() for k in ("x", "wg", "wu", "wd", "a", "u", "dout"))
    f, df = _act(a, st["act"])
    dh = torch.matmul(dout, wd)
    dwd = torch.matmul(dout.T, f * u)
    du = dh * f
    da = dh * u * df
    dx = torch.matmul(da, wg) + torch.matmul(du, wu)
    return tuple(t.to(torch.bfloat16) for t in (dx, torch.matmul(da.T, x), torch.matmul(du.T, x), dwd))


def _clip(st):
    grads = st["grads"]
    norm = torch.sqrt(torch.stack([torch.sum(g.float().double() ** 2) for g in grads]).sum()).float()
    by = torch.clamp(st["most"] / (norm + 1e-6), max=1.0)
    return norm, [(g.float() * by).to(g.dtype) for g in grads]


def _buckets(st):
    """[B or 1, Nq, Nk] whole numbers."""
    q = torch.arange(st["Nq"], device="cuda")[None] if st["posq"] is None else st["posq"].long()
    k = torch.arange(st["Nk"], device="cuda")[None] if st["posk"] is None else st["posk"].long()
    far = k[:, None, :] - q[:, :, None]
    starts = torch.tensor(st["starts"], device="cuda")
    n = far.abs() if st["two"] else (-far).clamp(min=0)
    at = torch.bucketize(n, starts, right=True) - 1
    return at + (far > 0) * len(st["starts"]) if st["two"] else at


def _relpos_fwd(st):
    bias = st["table"][_buckets(st)].permute(0, 3, 1, 2)
    if st["base"] is not None:
        bias = bias + st["base"].float()
    return bias.to(torch.bfloat16).expand(st["B"], -1, -1, -1).contiguous()


def _relpos_bwd(st):
    d = st["dbias"]
    B, H = d.shape[:2]
    at = _buckets(st).expand(B, -1, -1).reshape(-1)
    d = d.float().double().permute(0, 2, 3, 1).reshape(-1, H)
    return torch.zeros(st["table"].shape, dtype=torch.float64, device="cuda").index_add_(0, at, d).float()


def _run_plain(st):
    op = st["op"]
    if op == "rms_fwd":
        y, rstd, r = _rms_fwd(st["x"], st["gamma"], st["residual"])
        y = (_eight_bits(y) if st["bits8"] else y).to(st["x"].dtype)
        return (y, rstd) if st["residual"] is None else (y, rstd, r)
    return {"rms_bwd": _rms_bwd, "ffn_fwd": _ffn_fwd, "ffn_bwd": _ffn_bwd, "clip": _clip, "relpos_fwd": _relpos_fwd,
            "relpos_bwd": _relpos_bwd}[op](st)


# ------------------------------------------------------------------------------------------------ the framework's calls

def _run_own(st):
    from bwd_tri_attn_gb300 import binding as tb

    op = st["op"]
    if op == "rms_fwd":
        got = tb.rms_forward(st["x"], st["gamma"], st["residual"], eps=EPS, eight_bits="only" if st["bits8"] else False)
        y = tb.checkpoint_unpack(got.y8, dtype=st["x"].dtype) if st["bits8"] else got.y
        return (y, got.rstd) if st["residual"] is None else (y, got.rstd, got.r)
    if op == "rms_bwd":
        return tb.rms_backward(st["x"], st["gamma"], st["rstd"], st["dy"], dr=st["dr"])
    if op == "ffn_fwd":
        return tb.ffn_forward(st["x"], st["wg"], st["wu"], st["wd"], act=st["act"], keep=st["keep"])
    if op == "ffn_bwd":
        return tb.ffn_backward(st["x"], st["wg"], st["wu"], st["wd"], st["a"], st["u"], st["dout"], act=st["act"])
    if op == "clip":
        return tb.clip_gradients(st["grads"], st["most"], out=st["out"]), st["out"]
    if op == "relpos_fwd":
        return tb.relpos_forward(st["table"], st["starts"], st["Nq"], st["Nk"], B=st["B"], two_sided=st["two"], base=st["base"],
                                 positions=st["posq"], key_positions=st["posk"])
    return tb.relpos_backward(st["dbias"], st["starts"], two_sided=st["two"], positions=st["posq"], key_positions=st["posk"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------ 64-bit definition

def _exact_values(y):
    """What y (64 bits) kept in 8 bits stands for: the scale, its inverse and the scaled value are FP32 numbers by definition."""
    out = torch.zeros_like(y)
    for c in range(0, y.shape[1], GROUP):
        part = y[:, c:c + GROUP]
        top = part.abs().max(1).values
        top[top < TINY] = 0.0
        s = (top / 127.0).float().double()
        inv = torch.where(top > 0, 127.0 / top, torch.zeros_like(top)).float().double()
        scaled = (part * inv.unsqueeze(1)).float().double()
        out[:, c:c + GROUP] = torch.clamp(torch.round(scaled), -127, 127) * s.unsqueeze(1)
    return out


def _exact_gate(a, act):
    if act == "gelu":
        return 0.5 * a * torch.erfc(-a / 2 ** 0.5)
    return torch.sigmoid(a) if act == "sigmoid" else torch.nn.functional.silu(a)


def _exact_slope(a, act):
    if act == "gelu":
        return 0.5 * torch.erfc(-a / 2 ** 0.5) + a * torch.exp(torch.distributions.Normal(0.0, 1.0).log_prob(a))
    s = torch.sigmoid(a)
    return s * torch.sigmoid(-a) if act == "sigmoid" else s + a * s * torch.sigmoid(-a)


def _exact_relpos(st, case, backward):
    K = len(st["starts"])
    B, H, Nq, Nk = (case[k] for k in ("B", "H", "Nq", "Nk"))
    if backward:
        out = torch.zeros(st["table"].shape, dtype=torch.float64, device="cuda")
    else:
        out = torch.empty((B, H, Nq, Nk), dtype=torch.float64, device="cuda")
    for b in range(B):
        q = torch.arange(Nq, device="cuda") if st["posq"] is None else st["posq"][b].long()
        k = torch.arange(Nk, device="cuda") if st["posk"] is None else st["posk"][b].long()
        ahead = k.unsqueeze(0) - q.unsqueeze(1)
        if case["two"]:
            n, side = ahead.abs(), torch.where(ahead > 0, K, 0)
        else:
            n, side = torch.where(ahead < 0, -ahead, 0), torch.zeros_like(ahead)
        row = side - 1
        for s in st["starts"]:
            row = row + (n >= s).long()
        if not backward:
            for h in range(H):
                out[b, h] = st["table"][:, h].double()[row] + (0.0 if st["base"] is None else st["base"][b, h].double())
            continue
        for t in range(out.shape[0]):
            i, j = torch.nonzero(row == t, as_tuple=True)
            out[t] += st["dbias"][b][:, i, j].double().sum(1)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rms_fwd":
        x, total = st["x"], st["x"].double()
        r = total
        if st["residual"] is not None:
            total = total + st["residual"].double()
            r = total.float().to(x.dtype).double()  # (the norm is that of the rounded sum)
        rstd = torch.rsqrt(torch.linalg.vector_norm(r, dim=1) ** 2 / r.shape[1] + EPS)
        y = torch.einsum("mc,m,c->mc", r, rstd, st["gamma"].double())
        y = _exact_values(y) if case["bits8"] else y
        return (y, rstd) if st["residual"] is None else (y, rstd, total)
    if op == "rms_bwd":
        r, dy, rstd = st["x"].double(), st["dy"].double(), st["rstd"].double()
        g = dy * st["gamma"].double()
        along = torch.einsum("mc,mc->m", g, r) * rstd ** 3 / r.shape[1]
        dx = g * rstd.unsqueeze(1) - r * along.unsqueeze(1)
        return dx if st["dr"] is None else dx + st["dr"].double(), torch.einsum("mc,mc,m->c", dy, r, rstd)
    if op == "ffn_fwd":
        x = st["x"].double()
        a, u = x @ st["wg"].double().T, x @ st["wu"].double().T
        out = (_exact_gate(a, st["act"]) * u) @ st["wd"].double().T
        return (out, a, u) if case["keep"] else out
    if op == "ffn_bwd":
        a, u, dout = (st[k].double() for k in ("a", "u", "dout"))
        dh = dout @ st["wd"].double()
        x, wide = st["x"].double(), torch.cat([dh * u * _exact_slope(a, st["act"]), dh * _exact_gate(a, st["act"])], 1)
        dx = wide @ torch.cat([st["wg"], st["wu"]]).double()
        dw = wide.T @ x
        return dx, dw[:a.shape[1]], dw[a.shape[1]:], dout.T @ (_exact_gate(a, st["act"]) * u)
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in st["grads"]))
        by = min(1.0, st["most"] / (norm + 1e-6))
        return torch.tensor(norm, dtype=torch.float64), [g.double() * by for g in st["grads"]]
    return _exact_relpos(st, case, op == "relpos_bwd")
