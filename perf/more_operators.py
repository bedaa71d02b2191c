"""Measured cases of the gated delta rule (forward, backward, one token) and of the group norm with an activation,
channels last (forward, backward), which follows the heads of such a layer.

``own`` selects what ``run`` calls: the plain forms below (elementary torch operations in fp32, rounded once at the
end), or the framework's entry points.  ``exact`` gives the same outputs in fp64, token by token, written apart from
the plain forms.  Sizes follow the framework's workloads (8, 16, 32 heads of 128 channels, 2048 to 65536 tokens).
"""
import math
import random

import torch
import torch.nn.functional as F

own = False

EPS = 1e-5
CHUNK = 64
TYPES = {   # inputs (and their gradients), output; gates and write strengths are fp32
    "f32": (torch.float32, torch.float32),
    "bf16": (torch.bfloat16, torch.bfloat16),
    "f16": (torch.float16, torch.float16),
    "bf16_o32": (torch.bfloat16, torch.float32),
}


# ---------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a training step's delta layer at the framework's ordinary workload (4 x 2048 tokens, 8 heads)
        dict(name="delta_fwd_b4_t2k_h8", op="delta_fwd", types="bf16", B=4, T=2048, H=8, HV=8, K=128, V=128, h0=True, pack=0),
        # packed batch, 16 documents of 128 to 8192 tokens, two value heads for each key head
        dict(name="delta_fwd_pack16_h16", op="delta_fwd", types="bf16_o32", B=16, T=8192, H=8, HV=16, K=128, V=128, h0=True, pack=1003),
        # prefill of one long context
        dict(name="delta_fwd_long_t64k_h32", op="delta_fwd", types="bf16", B=1, T=65536, H=32, HV=32, K=128, V=128, h0=False, pack=0),
        # a small fp32 model with sizes that divide nothing
        dict(name="delta_fwd_b3_t1001_h5", op="delta_fwd", types="f32", B=3, T=1001, H=5, HV=5, K=96, V=80, h0=True, pack=0),
        # the gradient at the ordinary workload
        dict(name="delta_bwd_b4_t2k_h8", op="delta_bwd", types="bf16", B=4, T=2048, H=8, HV=8, K=128, V=128, h0=True, pack=0),
        # the gradient of a packed batch of 8 documents, four value heads for each key head
        dict(name="delta_bwd_pack8_h16", op="delta_bwd", types="bf16", B=8, T=3500, H=4, HV=16, K=128, V=128, h0=False, pack=77),
        # serving: one token of one sequence through 8 heads (latency)
        dict(name="delta_step_b1_h8", op="delta_step", types="bf16", B=1, H=8, HV=8, K=128, V=128, pool=1),
        # serving: 128 running sequences, 32 value heads on 16 key heads (the states are all of the traffic)
        dict(name="delta_step_b128_h32", op="delta_step", types="bf16", B=128, H=16, HV=32, K=128, V=128, pool=160),
        # the heads of a mixing layer's output, token by token: 16 heads of 128
        dict(name="group_norm_fwd_tokens32k", op="group_norm_fwd", types="bf16", N=32768, S=1, C=2048, G=16, act="none"),
        # features of eight 64 x 64 maps, 32 groups of 16 channels, with SiLU
        dict(name="group_norm_fwd_maps8_c512", op="group_norm_fwd", types="bf16", N=8, S=4096, C=512, G=32, act="silu"),
        # the gradient of the same maps' norm in training
        dict(name="group_norm_bwd_maps8_c512", op="group_norm_bwd", types="bf16", N=8, S=4096, C=512, G=32, act="silu"),
        # a small fp32 model: three sequences of 1001 positions, 40 groups of 13 channels
        dict(name="group_norm_bwd_n3_s1001_c520", op="group_norm_bwd", types="f32", N=3, S=1001, C=520, G=40, act="silu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _head_sizes(rng):
    if rng.random() < 0.75:
        return rng.choice([64, 128]), rng.choice([64, 128, 256])
    return rng.randint(16, 256), rng.randint(16, 256)


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_bwd", "delta_step", "group_norm_fwd", "group_norm_bwd"])
    if op in ("delta_fwd", "delta_bwd"):
        types = rng.choice(list(TYPES) if op == "delta_fwd" else ["f32", "bf16", "f16"])
        K, V = _head_sizes(rng)
        # a share of the largest listed case's tokens times heads times state
        most = (65536 * 32 if op == "delta_fwd" else 200000) * 128 * 128 // (4 if types == "f32" else 1)
        H = _log_int(rng, 1, 32)
        HV = H * rng.choice([1, 1, 2, 4])
        T = max(1, min(_log_int(rng, 1, 65536 if op == "delta_fwd" else 16384), most // (HV * K * V)))
        B = max(1, min(_log_int(rng, 1, 16), most // (T * HV * K * V)))
        pack = rng.randrange(1, 1 << 20) if rng.random() < 0.3 else 0
        return dict(op=op, types=types, B=B, T=T, H=H, HV=HV, K=K, V=V, h0=rng.random() < 0.5, pack=pack)
    if op == "delta_step":
        B, H = _log_int(rng, 1, 128), _log_int(rng, 1, 16)
        K, V = _head_sizes(rng)
        HV = H * rng.choice([1, 1, 2])
        B = max(1, min(B, 128 * 32 * 128 * 128 // (HV * K * V)))
        return dict(op=op, types=rng.choice(list(TYPES)), B=B, H=H, HV=HV, K=K, V=V, pool=B + rng.randrange(0, 32))
    types = rng.choice(["f32", "bf16", "f16"])
    width = rng.choice([_log_int(rng, 1, 256), 64, 128])
    G = _log_int(rng, 1, 64)
    C = width * G
    S = 1 if rng.random() < 0.4 else _log_int(rng, 1, 16384)
    S = max(1, min(S, (1 << 25) // C))
    N = max(1, min(_log_int(rng, 1, 65536 if S == 1 else 64), (1 << 26) // (S * C)))
    return dict(op=op, types=types, N=N, S=S, C=C, G=G, act=rng.choice(["none", "silu"]))


def _lengths(case):
    """Sequence lengths: B times T, or with ``pack`` B lengths drawn from [T / 64, T]."""
    if not case["pack"]:
        return [case["T"]] * case["B"]
    r = random.Random(case["pack"])
    return [r.randint(case["T"] // 64, case["T"]) for _ in range(case["B"])]


def work(case):
    op, (tx, to) = case["op"], TYPES[case["types"]]
    if op in ("group_norm_fwd", "group_norm_bwd"):
        n = case["N"] * case["S"] * case["C"]
        stats = 8 * case["N"] * case["G"]
        if op == "group_norm_fwd":
            return dict(bytes=2 * n * tx.itemsize + stats + 8 * case["C"], flops=10 * n)
        return dict(bytes=3 * n * tx.itemsize + stats + 16 * case["C"], flops=20 * n)
    H, HV, K, V = (case[k] for k in ("H", "HV", "K", "V"))
    if op == "delta_step":
        return dict(bytes=case["B"] * (8 * HV * K * V + 2 * H * K * tx.itemsize + HV * V * (tx.itemsize + to.itemsize) + 8 * HV),
                    flops=case["B"] * HV * 7 * K * V)
    rows, state = sum(_lengths(case)), 4 * case["B"] * HV * K * V
    if op == "delta_fwd":   # a token's products: k S, k^T n, q S
        return dict(bytes=rows * (2 * H * K * tx.itemsize + HV * V * (tx.itemsize + to.itemsize) + 8 * HV) + state * (1 + case["h0"]),
                    flops=rows * HV * 6 * K * V)
    # reads q, k, v, do and gates, writes their gradients; 8 products a token (two of them the states again)
    return dict(bytes=rows * (4 * H * K * tx.itemsize + 3 * HV * V * tx.itemsize + 16 * HV) + state * (2 + case["h0"]),
                flops=rows * HV * 16 * K * V)


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)   # noqa: E731
    op, (tx, to) = case["op"], TYPES[case["types"]]
    s = dict(op=op, types=(tx, to), case=case)
    if op in ("group_norm_fwd", "group_norm_bwd"):
        N, S, C, G = (case[k] for k in ("N", "S", "C", "G"))
        shape = (N, C) if S == 1 else (N, S, C)
        s["x"] = (rand(*shape) * (1 + 0.2 * rand(C)) + 0.5 * rand(C)).to(tx)
        s["w"], s["b"] = 1 + 0.1 * rand(C), 0.1 * rand(C)
        s["act"] = None if case["act"] == "none" else case["act"]
        if op == "group_norm_bwd":   # the statistics that the forward has saved
            s["mean"], s["rstd"] = _statistics(s["x"].float(), G)
            s["dy"] = rand(*shape).to(tx)
        return s
    H, HV, K, V = (case[k] for k in ("H", "HV", "K", "V"))
    unit = lambda *shape: F.normalize(rand(*shape), dim=-1).to(tx)            # noqa: E731
    rate = 2.0 ** (-6 * torch.arange(HV, device="cuda") / HV)                 # heads that forget fast and slowly
    if op == "delta_step":
        B, S = case["B"], case["pool"]
        s["q"], s["k"], s["v"] = unit(B, H, K), unit(B, H, K), rand(B, HV, V).to(tx)
        s["g"], s["beta"] = F.logsigmoid(rand(B, HV)) * rate, rand(B, HV).sigmoid()
        s["state"], s["out"] = 0.5 * rand(S, HV, K, V), torch.zeros(S, HV, K, V, device="cuda")
        s["slots"] = torch.randperm(S, device="cuda", generator=gen)[:B].to(torch.int32)
        return s
    lengths = _lengths(case)
    rows = (1, sum(lengths)) if case["pack"] else (case["B"], case["T"])
    ends = torch.tensor([0] + lengths).cumsum(0)
    s["cu"] = ends.to(device="cuda", dtype=torch.int32) if case["pack"] else None
    # row of each sequence's token, padded to whole chunks with -1 (for the plain form and the definition)
    most = -(-max(lengths) // CHUNK) * CHUNK
    at = torch.arange(most)[None].expand(len(lengths), -1)
    s["rows"] = torch.where(at < torch.tensor(lengths)[:, None], at + ends[:-1, None], -1).cuda()
    s["q"], s["k"], s["v"] = unit(*rows, H, K), unit(*rows, H, K), rand(*rows, HV, V).to(tx)
    s["g"], s["beta"] = F.logsigmoid(rand(*rows, HV)) * rate, rand(*rows, HV).sigmoid()
    s["h0"] = 0.5 * rand(len(lengths), HV, K, V) if case["h0"] else None
    if op == "delta_bwd":
        s["do"], s["dht"] = rand(*rows, HV, V).to(tx), 0.5 * rand(len(lengths), HV, K, V)
    return s


# ---------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------

def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _chunked(s, name):
    """An input's rows as [N, heads, chunks, CHUNK, ...] in fp32, zeros behind a sequence's end; key heads repeated."""
    t = s[name]
    heads, rows = t.shape[2], s["rows"]
    t = t.reshape(-1, *t.shape[2:])[rows.clamp_min(0)].float()
    t = t * (rows >= 0).reshape(*rows.shape, *[1] * (t.dim() - 2))
    t = t.repeat_interleave(s["v"].shape[2] // heads, 2).transpose(1, 2)
    return t.reshape(t.shape[0], t.shape[1], -1, CHUNK, *t.shape[3:])


def _unchunked(s, t, like, dtype):
    """The rows of [N, heads, chunks, CHUNK, ...] where input ``like`` has them, heads summed over those that share."""
    shape, rows = s[like].shape, s["rows"]
    t = t.reshape(t.shape[0], t.shape[1], -1, *t.shape[4:]).transpose(1, 2)
    if shape[2] != t.shape[2]:
        t = t.reshape(*t.shape[:2], shape[2], -1, t.shape[-1]).sum(3)
    return t[rows >= 0].reshape(*shape[:2], *t.shape[2:]).to(dtype)


def _delta_chunks(s):
    """What a chunk's products need: q, k, v, beta, and the decays from the start, between rows, to the end."""
    q, k, v, beta = (_chunked(s, n) for n in ("q", "k", "v", "beta"))
    G = _chunked(s, "g").double().cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = (G[..., :, None] - G[..., None, :]).masked_fill(~lower, -math.inf).exp().float()
    start, end = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None]
    kk = (k @ k.transpose(-1, -2)) * decay * beta[..., None]
    inverse = torch.eye(CHUNK, device=q.device).expand(kk.shape).clone()   # of I + tril(kk, -1), row by row
    for i in range(1, CHUNK):
        inverse[..., i, :i] = -(kk[..., i, None, :i] @ inverse[..., :i, :i])[..., 0, :]
    scores = (q @ k.transpose(-1, -2)) * decay
    return q, k, v, beta[..., None], decay, start, end, inverse, scores


def _delta_states(s, c):
    """States at the chunks' starts, update rows of the tokens, and the state at the end."""
    q, k, v, beta, decay, start, end, inverse, scores = c
    u, w, last = inverse @ (beta * v), inverse @ (beta * start * k), start[..., -1:, :]
    S = torch.zeros(*u.shape[:2], q.shape[-1], v.shape[-1], device=q.device) if s["h0"] is None else s["h0"]
    states, rows = [], []
    for i in range(u.shape[2]):
        states.append(S)
        rows.append(u[:, :, i] - w[:, :, i] @ S)
        S = last[:, :, i] * S + (end[:, :, i] * k[:, :, i]).transpose(-1, -2) @ rows[-1]
    return torch.stack(states, 2), torch.stack(rows, 2), S


def _delta_fwd(s):
    c = _delta_chunks(s)
    q, start, scores = c[0], c[5], c[8]
    states, rows, S = _delta_states(s, c)
    o = ((start * q) @ states + scores @ rows) * q.shape[-1] ** -0.5
    return _unchunked(s, o, "v", s["types"][1]), S


def _delta_bwd(s):
    c = _delta_chunks(s)
    q, k, v, beta, decay, start, end, inverse, scores = c
    states, rows, _ = _delta_states(s, c)
    do = _chunked(s, "do") * q.shape[-1] ** -0.5
    last, turn = start[..., -1:, :], lambda t: t.transpose(-1, -2)   # noqa: E731
    local = turn(scores) @ do
    dS, dstates, dx = s["dht"], [None] * q.shape[2], [None] * q.shape[2]
    for i in range(q.shape[2] - 1, -1, -1):
        dstates[i] = dS
        dx[i] = turn(inverse[:, :, i]) @ (local[:, :, i] + (end[:, :, i] * k[:, :, i]) @ dS)
        dS = last[:, :, i] * dS + turn(start[:, :, i] * q[:, :, i]) @ do[:, :, i] - \
            turn(beta[:, :, i] * start[:, :, i] * k[:, :, i]) @ dx[i]
    dstates, dx = torch.stack(dstates, 2), torch.stack(dx, 2)
    dscores = (do @ turn(rows)) * decay
    dinner = -(dx @ turn(rows)).tril(-1) * decay
    dq = start * (do @ turn(states)) + dscores @ k
    drow = dinner @ k - start * (dx @ turn(states))
    dcol = turn(dscores) @ q + turn(beta * dinner) @ k + end * (rows @ turn(dstates))
    dk = beta * drow + dcol
    dbeta = (dx * v).sum(-1) + (k * drow).sum(-1)
    dG = ((q * dq).sum(-1) + beta[..., 0] * (k * drow).sum(-1) - (k * dcol).sum(-1)).double()
    at_end = (last[..., None, 0, 0] * (states * dstates).sum((-1, -2))[..., None])[..., 0] + \
        ((end * (rows @ turn(dstates))) * k).sum((-1, -2))
    dG[..., -1] += at_end.double()
    dg = dG.flip(-1).cumsum(-1).flip(-1).float()
    tx = s["types"][0]
    return (_unchunked(s, dq, "q", tx), _unchunked(s, dk, "k", tx), _unchunked(s, beta * dx, "v", tx),
            _unchunked(s, dg[..., None], "g", torch.float32)[..., 0], _unchunked(s, dbeta[..., None], "beta", torch.float32)[..., 0], dS)


def _delta_step(s):
    at, per = s["slots"].long(), s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(per, 1) for n in ("q", "k"))
    old = s["g"].exp()[..., None, None] * s["state"][at]
    row = s["beta"][..., None] * (s["v"].float() - (k[..., None] * old).sum(-2))
    new = old + k[..., None] * row[..., None, :]
    s["out"][at] = new
    return (q[..., None] * new).sum(-2).mul(q.shape[-1] ** -0.5).to(s["types"][1]), s["out"]


def _statistics(x, groups):
    parts = x.reshape(x.shape[0], -1, groups, x.shape[-1] // groups)
    mean = parts.mean((1, 3))
    var = (parts - mean[:, None, :, None]).square().mean((1, 3))
    return mean, (var + EPS).rsqrt()


def _normed(x, mean, rstd):
    parts = x.reshape(x.shape[0], -1, mean.shape[1], x.shape[-1] // mean.shape[1])
    return ((parts - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)


def _group_norm_fwd(s):
    x = s["x"].float()
    mean, rstd = _statistics(x, s["case"]["G"])
    z = _normed(x, mean, rstd) * s["w"] + s["b"]
    y = z if s["act"] is None else z / (1 + (-z).exp())
    return y.to(s["types"][0]), mean, rstd


def _group_norm_bwd(s):
    n, dz = _normed(s["x"].float(), s["mean"], s["rstd"]), s["dy"].float()
    if s["act"] is not None:
        z = n * s["w"] + s["b"]
        sig = 1 / (1 + (-z).exp())
        dz = dz * sig * (1 + z * (1 - sig))
    G = s["case"]["G"]
    parts = lambda t: t.reshape(t.shape[0], -1, G, t.shape[-1] // G)   # noqa: E731
    a, p = parts(dz * s["w"]), parts(n)
    dx = (a - a.mean((1, 3), keepdim=True) - p * (a * p).mean((1, 3), keepdim=True)) * s["rstd"][:, None, :, None]
    over = tuple(range(n.dim() - 1))
    return dx.reshape(n.shape).to(s["types"][0]), (dz * n).sum(over), dz.sum(over)


_PLAIN = dict(delta_fwd=_delta_fwd, delta_bwd=_delta_bwd, delta_step=_delta_step, group_norm_fwd=_group_norm_fwd,
              group_norm_bwd=_group_norm_bwd)


def _binding():
    from chunkwise_gated_linear_chunked_gb300 import binding
    return binding


def _own_delta_fwd(s):
    return _binding().delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], initial_state=s["h0"], cu_seqlens=s["cu"],
                                out_dtype=s["types"][1])


def _own_delta_bwd(s):
    return _binding().delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], initial_state=s["h0"], dht=s["dht"],
                                cu_seqlens=s["cu"])


def _own_delta_step(s):
    o = _binding().delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"], state_out=s["out"],
                              out_dtype=s["types"][1])
    return o, s["out"]


def _own_group_norm_fwd(s):
    return _binding().group_norm_fwd(s["x"], s["case"]["G"], weight=s["w"], bias=s["b"], activation=s["act"], eps=EPS)


def _own_group_norm_bwd(s):
    return _binding().group_norm_bwd(s["x"], s["mean"], s["rstd"], s["dy"], weight=s["w"], bias=s["b"], activation=s["act"])


_OWN = dict(delta_fwd=_own_delta_fwd, delta_bwd=_own_delta_bwd, delta_step=_own_delta_step,
            group_norm_fwd=_own_group_norm_fwd, group_norm_bwd=_own_group_norm_bwd)


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if case["op"] == "delta_step":
        out, o, per = wide["out"], [], case["HV"] // case["H"]
        for b, slot in enumerate(s["slots"].tolist()):
            heads = []
            for h in range(case["HV"]):
                S = torch.exp(wide["g"][b, h]) * wide["state"][slot, h]
                k, q = wide["k"][b, h // per], wide["q"][b, h // per]
                out[slot, h] = S + torch.outer(k, wide["beta"][b, h] * (wide["v"][b, h] - k @ S))
                heads.append(q @ out[slot, h] / math.sqrt(case["K"]))
            o.append(torch.stack(heads))
        return torch.stack(o), out
    if case["op"] == "delta_fwd":
        return _Steps(s, wide).forward()
    if case["op"] == "delta_bwd":
        return _Steps(s, wide).backward()
    return _exact_group_norm(case, wide)


class _Steps:
    """The recurrence over tokens, all sequences and value heads side by side, in fp64."""

    def __init__(self, s, wide):
        self.s, self.at = s, s["rows"].T.contiguous()      # [steps, N]
        self.live = self.at >= 0
        self.wide, self.per = wide, s["v"].shape[2] // s["q"].shape[2]
        self.flat = {n: wide[n].reshape(-1, *wide[n].shape[2:]) for n in ("q", "k", "v", "g", "beta", "do") if n in wide}
        self.scale = s["q"].shape[-1] ** -0.5
        N, HV, K, V = s["rows"].shape[0], s["v"].shape[2], s["q"].shape[3], s["v"].shape[3]
        self.zero = torch.zeros(N, HV, K, V, dtype=torch.float64, device=s["q"].device)

    def token(self, t, *names):
        """Rows of step t; behind a sequence's end they are zeros, which leave its state as it is."""
        out = []
        for n in names:
            r = self.flat[n][self.at[t].clamp_min(0)]
            r = torch.where(self.live[t].reshape(-1, *[1] * (r.dim() - 1)), r, torch.zeros_like(r))
            out.append(r.repeat_interleave(self.per, 1) if n in ("q", "k") else r)
        return out

    def advance(self, t, S):
        k, v, g, beta = self.token(t, "k", "v", "g", "beta")
        S = S * g.exp()[..., None, None]
        row = beta[..., None] * (v - torch.einsum("nhk,nhkv->nhv", k, S))
        return torch.baddbmm(S.flatten(0, 1), k.flatten(0, 1)[:, :, None], row.flatten(0, 1)[:, None, :]).view_as(S), row

    def put(self, dest, t, value):
        """Adds a step's rows to a gradient, heads of one key head together."""
        live = self.live[t]
        if value.shape[1] != dest.shape[1]:
            value = value.reshape(value.shape[0], dest.shape[1], self.per, -1).sum(2)
        dest[self.at[t][live]] = value[live]

    def forward(self):
        S = self.wide["h0"] if self.s["h0"] is not None else self.zero
        o = torch.empty_like(self.flat["v"])
        for t in range(self.at.shape[0]):
            S, _ = self.advance(t, S)
            q, = self.token(t, "q")
            self.put(o, t, self.scale * torch.einsum("nhk,nhkv->nhv", q, S))
        return o.view_as(self.wide["v"]), S

    def backward(self, block=64):
        S = self.wide["h0"] if self.s["h0"] is not None else self.zero
        starts = []
        for t in range(self.at.shape[0]):
            if t % block == 0:
                starts.append(S)
            S, _ = self.advance(t, S)
        d = {n: torch.empty_like(self.flat[n]) for n in ("q", "k", "v", "g", "beta")}
        dS = self.wide["dht"]
        for b in range(len(starts) - 1, -1, -1):
            kept, S = [], starts[b]
            span = range(b * block, min((b + 1) * block, self.at.shape[0]))
            for t in span:
                new, row = self.advance(t, S)
                kept.append((S, new, row))
                S = new
            for t in reversed(span):
                q, k, v, g, beta, do = self.token(t, "q", "k", "v", "g", "beta", "do")
                S, new, row = kept.pop()
                S, do = S * g.exp()[..., None, None], self.scale * do
                dS = dS + q[..., None] * do[..., None, :]
                drow = torch.einsum("nhk,nhkv->nhv", k, dS)
                back = beta[..., None] * drow
                self.put(d["q"], t, torch.einsum("nhkv,nhv->nhk", new, do))
                self.put(d["k"], t, torch.einsum("nhkv,nhv->nhk", dS, row) - torch.einsum("nhkv,nhv->nhk", S, back))
                self.put(d["v"], t, back)
                self.put(d["beta"], t, (drow * (v - torch.einsum("nhk,nhkv->nhv", k, S))).sum(-1))
                dS = dS - k[..., None] * back[..., None, :]
                self.put(d["g"], t, (dS * S).sum((-1, -2)))
                dS = dS * g.exp()[..., None, None]
        return tuple(d[n].reshape(self.wide[n].shape) for n in ("q", "k", "v", "g", "beta")) + (dS,)


def _exact_group_norm(case, wide):
    N, S, C, G = (case[k] for k in ("N", "S", "C", "G"))
    cut = lambda t: t.reshape(N, S, G, C // G).permute(0, 2, 1, 3).reshape(N, G, S * (C // G))             # noqa: E731
    join = lambda t: t.reshape(N, G, S, C // G).permute(0, 2, 1, 3).reshape(wide["x"].shape)              # noqa: E731
    x, w, b, silu = cut(wide["x"]), wide["w"], wide["b"], case["act"] == "silu"
    if case["op"] == "group_norm_fwd":
        mean = x.sum(-1) / x.shape[-1]
        x = x - mean[..., None]
        rstd = 1 / torch.sqrt(torch.linalg.vector_norm(x, dim=-1) ** 2 / x.shape[-1] + EPS)
        z = torch.addcmul(b, join(x * rstd[..., None]), w)
        return z * torch.sigmoid(z) if silu else z, mean, rstd
    mean, rstd = wide["mean"], wide["rstd"]
    n = (x - mean[..., None]) * rstd[..., None]
    dz = wide["dy"]
    if silu:
        z = torch.addcmul(b, join(n), w)
        sig = torch.sigmoid(z)
        dz = dz * (sig + z * sig * (1 - sig))
    a = cut(dz * w)
    inner = torch.einsum("ngi,ngi->ng", a, n)
    dx = rstd[..., None] * (a - (a.sum(-1)[..., None] + n * inner[..., None]) / x.shape[-1])
    flat = lambda t: t.reshape(-1, C)                                                                      # noqa: E731
    return join(dx), torch.einsum("rc,rc->c", flat(dz), flat(join(n))), flat(dz).sum(0)
