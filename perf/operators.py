"""Measured cases of the operators that stand beside the GLA kernels in a model: the gated linear recurrence
(forward, backward, one token), the GLA state update for one token, and the root-mean-square norm with the
residual's addition (forward in 16 or 32 bits, forward in 8 bits with scales, backward).

``own`` selects what ``run`` calls: the plain forms below (elementary torch operations in fp32, rounded once at
the end), or the framework's entry points.  ``exact`` gives the same outputs in fp64, written apart from the plain
forms.  Sizes follow the framework's workloads (H = 8, 16, 32 heads of 128 channels, T = 2048 to 65536 tokens).
"""
import math
import random

import torch
import torch.nn.functional as F

own = False

EPS = 1e-6
E4M3_MAX = 448.0
SCALE_MIN = 1e-30    # smallest scale of an 8-bit group (a group of zeros)
TYPES = {            # x (and the gradients of x), gate, output
    "f32": (torch.float32, torch.float32, torch.float32),
    "bf16": (torch.bfloat16, torch.bfloat16, torch.bfloat16),
    "f16": (torch.float16, torch.float16, torch.float16),
    "bf16_o32": (torch.bfloat16, torch.bfloat16, torch.float32),
    "bf16_gf32": (torch.bfloat16, torch.float32, torch.float32),
}


# ---------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a training step's recurrent layer at the framework's ordinary workload (4 x 2048 tokens, 8 heads)
        dict(name="scan_fwd_b4_t2k_d1024", op="scan_fwd", types="bf16", B=4, T=2048, D=1024, h0=True, pack=0),
        # prefill of one long context: few sequences, so the time axis itself has to be split
        dict(name="scan_fwd_long_t64k_d4096", op="scan_fwd", types="bf16", B=1, T=65536, D=4096, h0=False, pack=0),
        # packed training batch, 16 documents of 128 to 8192 tokens, gates kept in fp32
        dict(name="scan_fwd_pack16_d2048", op="scan_fwd", types="bf16_gf32", B=16, T=8192, D=2048, h0=True, pack=1003),
        # the gradient of a recurrent layer in training
        dict(name="scan_bwd_b8_t4k_d2048", op="scan_bwd", types="bf16", B=8, T=4096, D=2048, h0=True, pack=0),
        # a small fp32 model with sizes that divide nothing
        dict(name="scan_bwd_b3_t1000_d1001", op="scan_bwd", types="f32", B=3, T=1000, D=1001, h0=True, pack=0),
        # serving: one token for each of 64 running sequences, states in a pool
        dict(name="scan_step_b64_d4096", op="scan_step", types="bf16", B=64, D=4096, pool=96),
        # serving: one token of one sequence through a GLA layer of 8 heads (latency)
        dict(name="gla_step_b1_h8", op="gla_step", types="bf16", B=1, H=8, K=128, V=128, pool=1),
        # serving: 128 running sequences, 16 heads with wide values (the states are all of the traffic)
        dict(name="gla_step_b128_h16_v256", op="gla_step", types="bf16", B=128, H=16, K=128, V=256, pool=160),
        # pre-norm of the next block over a long context
        dict(name="norm_fwd_t64k_d4096", op="norm_fwd", types="bf16", rows=65536, D=4096, residual="same"),
        # serving: the norm of one token, in 8 bits for the next projection (latency)
        dict(name="norm_quant_r1_d2048", op="norm_quant", types="bf16", rows=1, D=2048, residual="same", group=0),
        # training with an fp32 residual stream and 8-bit activations in groups of 128
        dict(name="norm_quant_t16k_d2048", op="norm_quant", types="bf16", rows=16384, D=2048, residual="f32", group=128),
        # the norm's gradient in training
        dict(name="norm_bwd_t32k_d2048", op="norm_bwd", types="bf16", rows=32768, D=2048, residual="same"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_bwd", "scan_step", "gla_step", "norm_fwd", "norm_quant", "norm_bwd"])
    if op in ("scan_fwd", "scan_bwd"):
        types = rng.choice(list(TYPES))
        most = (1 << 28) * 3 // sum(t.itemsize for t in TYPES[types])   # rows times channels
        D = _log_int(rng, 64, 4096)
        if rng.random() < 0.5:
            D = max(64, D // 64 * 64)
        T = min(_log_int(rng, 1, 65536), most // D)
        B = max(1, min(_log_int(rng, 1, 64), most // (T * D)))
        pack = rng.randrange(1, 1 << 20) if rng.random() < 0.3 else 0
        return dict(op=op, types=types, B=B, T=T, D=D, h0=rng.random() < 0.5, pack=pack)
    if op == "scan_step":
        B = _log_int(rng, 1, 512)
        return dict(op=op, types=rng.choice(list(TYPES)), B=B, D=_log_int(rng, 64, 8192), pool=B + rng.randrange(0, 64))
    if op == "gla_step":
        B = _log_int(rng, 1, 128)
        return dict(op=op, types=rng.choice(["f32", "bf16", "bf16_o32", "bf16_gf32"]), B=B, H=_log_int(rng, 1, 32),
                    K=rng.choice([64, 128]), V=rng.choice([64, 128, 256]), pool=B + rng.randrange(0, 32))
    types = rng.choice(["f32", "bf16", "f16"])
    D = _log_int(rng, 64, 8192)
    if rng.random() < 0.5:
        D = max(64, D // 64 * 64)
    rows = min(_log_int(rng, 1, 65536), (1 << 26) // D)
    case = dict(op=op, types=types, rows=rows, D=D, residual=rng.choice(["same", "f32"] + ["none"] * (op != "norm_bwd")))
    if op == "norm_quant":
        case["group"] = rng.choice([0, 128])
    return case


def _lengths(case):
    """Sequence lengths of a scan case: B times T, or with ``pack`` B lengths drawn from [T / 64, T]."""
    if not case["pack"]:
        return [case["T"]] * case["B"]
    r = random.Random(case["pack"])
    return [r.randint(case["T"] // 64, case["T"]) for _ in range(case["B"])]


def work(case):
    op, (tx, tg, to) = case["op"], TYPES[case["types"]]
    if op in ("scan_fwd", "scan_bwd"):
        n = sum(_lengths(case)) * case["D"]
        state = 4 * case["B"] * case["D"]
        if op == "scan_fwd":
            return dict(bytes=n * (tx.itemsize + tg.itemsize + to.itemsize) + state * (1 + case["h0"]), flops=3 * n)
        # reads g, h, dh (and h0, dht); writes dx, dg (and dh0)
        return dict(bytes=n * (2 * tg.itemsize + 2 * to.itemsize + tx.itemsize) + state * (2 + case["h0"]), flops=4 * n)
    if op == "scan_step":
        n = case["B"] * case["D"]
        return dict(bytes=n * (tx.itemsize + tg.itemsize + to.itemsize + 8), flops=3 * n)
    if op == "gla_step":
        n = case["B"] * case["H"]
        K, V = case["K"], case["V"]
        return dict(bytes=n * (8 * K * V + 2 * K * tx.itemsize + K * tg.itemsize + V * (tx.itemsize + to.itemsize)),
                    flops=n * 5 * K * V)
    rows, D = case["rows"], case["D"]
    tr = torch.float32 if case["residual"] == "f32" else tx
    if op == "norm_bwd":   # reads s, dy, ds, rstd, w; writes the gradients of x and of the residual, and dw
        out = tr.itemsize if tr == tx else tr.itemsize + tx.itemsize
        return dict(bytes=rows * D * (2 * tr.itemsize + tx.itemsize + out) + 4 * rows + 8 * D, flops=10 * rows * D)
    res = 0 if case["residual"] == "none" else 2 * tr.itemsize
    out = tx.itemsize if op == "norm_fwd" else 1
    extra = 4 * rows * (1 if op == "norm_fwd" else 1 + _groups(case))
    return dict(bytes=rows * D * (tx.itemsize + res + out) + extra + 4 * D, flops=5 * rows * D)


def _groups(case):
    return -(-case["D"] // case["group"]) if case["group"] else 1


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    gate = lambda *shape: F.logsigmoid(rand(*shape)) / 16                    # noqa: E731
    op, (tx, tg, to) = case["op"], TYPES[case["types"]]
    s = dict(op=op, types=(tx, tg, to), case=case)
    if op in ("scan_fwd", "scan_bwd"):
        D, lengths = case["D"], _lengths(case)
        shape = (1, sum(lengths), D) if case["pack"] else (case["B"], case["T"], D)
        ends = torch.tensor([0] + lengths).cumsum(0)
        s["cu"] = ends.to(device="cuda", dtype=torch.int32) if case["pack"] else None
        s["ends"] = ends.cuda()
        s["x"], s["g"] = rand(*shape).to(tx), gate(*shape).to(tg)
        s["h0"] = 0.5 * rand(len(lengths), D) if case["h0"] else None
        if op == "scan_bwd":   # the forward's output, as a training step has saved it
            s["h"] = _scan_fwd(s)[0]
            s["dh"], s["dht"] = rand(*shape).to(to), rand(len(lengths), D)
            del s["x"]
    elif op == "scan_step":
        B, D, S = case["B"], case["D"], case["pool"]
        s["x"], s["g"] = rand(B, D).to(tx), gate(B, D).to(tg)
        s["state"], s["out"] = 0.5 * rand(S, D), torch.zeros(S, D, device="cuda")
        s["slots"] = torch.randperm(S, device="cuda", generator=gen)[:B].to(torch.int32)
    elif op == "gla_step":
        B, H, K, V, S = (case[k] for k in ("B", "H", "K", "V", "pool"))
        s["q"], s["k"], s["v"] = rand(B, H, K).to(tx), rand(B, H, K).to(tx), rand(B, H, V).to(tx)
        s["g"] = gate(B, H, K).to(tg)
        s["state"], s["out"] = rand(S, H, K, V), torch.zeros(S, H, K, V, device="cuda")
        s["slots"] = torch.randperm(S, device="cuda", generator=gen)[:B].to(torch.int32)
    else:
        rows, D = case["rows"], case["D"]
        tr = torch.float32 if case["residual"] == "f32" else tx
        s["w"] = 1 + 0.1 * rand(D)
        if op == "norm_bwd":
            s["s"] = (1.4 * rand(rows, D)).to(tr)
            s["rstd"] = (s["s"].float().square().mean(-1) + EPS).rsqrt()
            s["dy"], s["ds"] = rand(rows, D).to(tx), rand(rows, D).to(tr)
        else:
            s["x"] = rand(rows, D).to(tx)
            s["res"] = None if case["residual"] == "none" else rand(rows, D).to(tr)
            s["group"] = case.get("group")
    return s


# ---------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------

def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _linear_scan(a, b):
    """y_t = a_t y_{t-1} + b_t along dim 0 (y_{-1} = 0), by doubling: log2 T passes of products and sums."""
    a, b, step = a.clone(), b.clone(), 1
    while step < a.shape[0]:
        b[step:] += a[step:] * b[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return b


def _scan_fwd(s):
    to, ends = s["types"][2], s["ends"]
    D = s["x"].shape[-1]
    a, b = s["g"].float().exp().reshape(-1, D), s["x"].float().reshape(-1, D).clone()
    full = ends[1:] > ends[:-1]
    first, last = ends[:-1][full], ends[1:][full] - 1
    if s["h0"] is not None:
        b[first] += a[first] * s["h0"][full]
    a[first] = 0
    h = _linear_scan(a, b)
    ht = torch.zeros(ends.numel() - 1, D, device=h.device) if s["h0"] is None else s["h0"].clone()
    ht[full] = h[last]
    return h.reshape(s["x"].shape).to(to), ht


def _scan_bwd(s):
    (tx, tg, _), ends = s["types"], s["ends"]
    D = s["g"].shape[-1]
    a, h = s["g"].float().exp().reshape(-1, D), s["h"].float().reshape(-1, D)
    lam = s["dh"].float().reshape(-1, D).clone()
    full = ends[1:] > ends[:-1]
    first, last = ends[:-1][full], ends[1:][full] - 1
    lam[last] += s["dht"][full]
    later = torch.zeros_like(a)
    later[:-1] = a[1:]
    later[last] = 0
    lam = _linear_scan(later.flip(0), lam.flip(0)).flip(0)
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    prev[first] = 0 if s["h0"] is None else s["h0"][full]
    mu = lam * a
    dh0 = s["dht"].clone()
    dh0[full] = mu[first]
    shape = s["g"].shape
    return lam.reshape(shape).to(tx), (mu * prev).reshape(shape).to(tg), dh0


def _scan_step(s):
    at = s["slots"].long()
    new = s["g"].float().exp() * s["state"][at] + s["x"].float()
    s["out"][at] = new
    return new.to(s["types"][2]), s["out"]


def _gla_step(s):
    at = s["slots"].long()
    q, k, v, a = s["q"].float(), s["k"].float(), s["v"].float(), s["g"].float().exp()
    new = a[..., None] * s["state"][at] + k[..., None] * v[..., None, :]
    s["out"][at] = new
    return (q[..., None] * new).sum(-2).mul(q.shape[-1] ** -0.5).to(s["types"][2]), s["out"]


def _normed(s):
    """(sum with the residual, 1 / rms, normed and weighted), all in fp32."""
    total = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
    rstd = (total.square().mean(-1) + EPS).rsqrt()
    return total, rstd, total * rstd[:, None] * s["w"]


def _norm_fwd(s):
    total, rstd, y = _normed(s)
    return y.to(s["types"][0]), None if s["res"] is None else total.to(s["res"].dtype), rstd


def _norm_quant(s):
    total, rstd, y = _normed(s)
    rows, D = y.shape
    group = s["group"] or D
    parts = F.pad(y, (0, -D % group)).reshape(rows, -1, group)
    scales = (parts.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
    q = (parts / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).reshape(rows, -1)[:, :D].to(torch.float8_e4m3fn)
    return q, scales, None if s["res"] is None else total.to(s["res"].dtype), rstd


def _norm_bwd(s):
    n, rstd, dy = s["s"].float() * s["rstd"][:, None], s["rstd"][:, None], s["dy"].float()
    wdy = s["w"] * dy
    grad = rstd * (wdy - n * (wdy * n).mean(-1, keepdim=True)) + s["ds"].float()
    return grad.to(s["types"][0]), grad.to(s["s"].dtype), (dy * n).sum(0)


_PLAIN = dict(scan_fwd=_scan_fwd, scan_bwd=_scan_bwd, scan_step=_scan_step, gla_step=_gla_step,
              norm_fwd=_norm_fwd, norm_quant=_norm_quant, norm_bwd=_norm_bwd)


def _binding():
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


def _own_scan_fwd(s):
    return _binding().scan_fwd(s["x"], s["g"], initial_state=s["h0"], cu_seqlens=s["cu"], out_dtype=s["types"][2])


def _own_scan_bwd(s):
    return _binding().scan_bwd(s["g"], s["h"], s["dh"], initial_state=s["h0"], dht=s["dht"], cu_seqlens=s["cu"],
                               dx_dtype=s["types"][0])


def _own_scan_step(s):
    h = _binding().scan_step(s["x"], s["g"], s["state"], slots=s["slots"], state_out=s["out"], out_dtype=s["types"][2])
    return h, s["out"]


def _own_gla_step(s):
    o = _binding().gla_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"], state_out=s["out"],
                            out_dtype=s["types"][2])
    return o, s["out"]


def _own_norm_fwd(s):
    y, total, rstd = _binding().norm_fwd(s["x"], residual=s["res"], weight=s["w"], eps=EPS)
    return y, None if s["res"] is None else total, rstd


def _own_norm_quant(s):
    q, scales, total, rstd = _binding().norm_quant_fwd(s["x"], residual=s["res"], weight=s["w"], eps=EPS, group=s["group"])
    return q, scales, None if s["res"] is None else total, rstd


def _own_norm_bwd(s):
    return _binding().norm_bwd(s["s"], s["rstd"], s["dy"], weight=s["w"], ds=s["ds"])


_OWN = dict(scan_fwd=_own_scan_fwd, scan_bwd=_own_scan_bwd, scan_step=_own_scan_step, gla_step=_own_gla_step,
            norm_fwd=_own_norm_fwd, norm_quant=_own_norm_quant, norm_bwd=_own_norm_bwd)


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if case["op"] == "scan_fwd":
        return _exact_scan_fwd(s, wide)
    if case["op"] == "scan_bwd":
        return _exact_scan_bwd(s, wide)
    if case["op"] == "scan_step":
        rows = s["slots"].tolist()
        h = torch.stack([torch.exp(wide["g"][b]) * wide["state"][r] + wide["x"][b] for b, r in enumerate(rows)])
        out = wide["out"]
        for b, r in enumerate(rows):
            out[r] = h[b]
        return h, out
    if case["op"] == "gla_step":
        out, o = wide["out"], []
        for b, r in enumerate(s["slots"].tolist()):
            out[r] = torch.diag_embed(wide["g"][b].exp()) @ wide["state"][r] + torch.einsum("hk,hv->hkv", wide["k"][b], wide["v"][b])
            o.append(torch.einsum("hk,hkv->hv", wide["q"][b], out[r]) / math.sqrt(case["K"]))
        return torch.stack(o), out
    w, D = wide["w"], case["D"]
    if case["op"] == "norm_bwd":
        r = wide["rstd"].unsqueeze(1)
        inner = torch.einsum("rd,rd,d->r", wide["dy"], wide["s"], w).unsqueeze(1)
        grad = wide["ds"] + r * w * wide["dy"] - r ** 3 * wide["s"] * inner / D
        return grad, grad, torch.einsum("rd,rd,r->d", wide["dy"], wide["s"], wide["rstd"])
    total = wide["x"] if s["res"] is None else torch.add(wide["x"], wide["res"])
    rstd = 1 / torch.sqrt(torch.linalg.vector_norm(total, dim=1) ** 2 / D + EPS)
    y = torch.einsum("rd,r,d->rd", total, rstd, w)
    sums = None if s["res"] is None else total
    if case["op"] == "norm_fwd":
        return y, sums, rstd
    width = case["group"] or D
    cuts = list(range(0, D, width))
    scales = torch.stack([torch.clamp(y[:, c:c + width].abs().max(dim=1).values / E4M3_MAX, min=SCALE_MIN) for c in cuts], 1)
    return torch.cat([y[:, c:c + width] / scales[:, i:i + 1] for i, c in enumerate(cuts)], 1), scales, sums, rstd


def _bounds(s):
    ends = s["ends"].tolist()
    return list(zip(ends[:-1], ends[1:]))


def _exact_scan_fwd(s, wide):
    D = s["x"].shape[-1]
    if s["cu"] is None:   # all sequences of a dense batch step together
        a, x = wide["g"].exp_(), wide["x"]
        h = wide["h0"] if s["h0"] is not None else torch.zeros(x.shape[0], D, dtype=torch.float64, device=x.device)
        out = torch.empty_like(x)
        for t in range(x.shape[1]):
            h = torch.addcmul(x[:, t], a[:, t], h, out=out[:, t])
        return out, h.clone()
    a, x = wide["g"].exp_()[0], wide["x"][0]
    out, ht = torch.empty_like(x), torch.zeros(len(_bounds(s)), D, dtype=torch.float64, device=x.device)
    # a pack steps all its sequences together too: row i of every sequence longer than i
    starts = s["ends"][:-1]
    count = s["ends"][1:] - starts
    if s["h0"] is not None:
        ht.copy_(wide["h0"])
    order = count.argsort(descending=True)
    longer = count[order].tolist()
    h, n = ht[order], len(longer)
    for t in range(max(longer)):
        while n and longer[n - 1] <= t:
            n -= 1
        at = starts[order[:n]] + t
        h[:n] = a[at] * h[:n] + x[at]
        out[at] = h[:n]
    ht[order] = h
    return out[None], ht


def _exact_scan_bwd(s, wide):
    D = s["g"].shape[-1]
    a, h, dh = wide["g"].exp_().view(-1, D), wide["h"].view(-1, D), wide["dh"].view(-1, D)
    starts = s["ends"][:-1]
    count = s["ends"][1:] - starts
    order = count.argsort(descending=True)
    longer, begins = count[order].tolist(), starts[order]
    mu = wide["dht"][order]   # the gradient that reaches a sequence's state from its later rows
    h0 = wide["h0"][order] if s["h0"] is not None else torch.zeros_like(mu)
    dx, dg = torch.empty_like(dh), torch.empty_like(dh)
    n = 0
    for t in range(max(longer) - 1, -1, -1):
        while n < len(longer) and longer[n] > t:
            n += 1
        at = begins[:n] + t
        lam = dh[at] + mu[:n]
        mu[:n] = lam * a[at]
        dx[at], dg[at] = lam, mu[:n] * (h[at - 1] if t else h0[:n])
    dh0 = torch.empty_like(mu)
    dh0[order] = mu
    return dx.view(s["g"].shape), dg.view(s["g"].shape), dh0
