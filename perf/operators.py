"""What is measured of linear attention with one decay per head (chunked forward, its gradients,
the single-token step) and of the norm of queries and keys with the position rotation.

Linear attention, per sequence and head, with a fixed log-decay l <= 0 per head:

    S_t = e^l S_{t-1} + k_t v_t^T,      o_t = dk^{-1/2} S_t^T q_t

Norm and rotation, per token and head, over the d channels of a query or key x:

    n = x * rsqrt(sum x^2 [/ d] + eps) * w,     (y_a, y_b) = rotation of the pair (n_a, n_b) by pos * f_j

A case is a dict; "op" names the operator.  `run` is one call as a user makes it: the framework's
(`own`) or the same in elementary torch operations in fp32.  `exact` restates the definitions in
fp64 by other routes (the quadratic form; explicit 2 x 2 rotations).
"""
import math

import torch

own = False

CHUNK = 128   # tokens of a block of the plain form


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a short prompt of one user, a ragged length: latency
        dict(name="fwd_prompt_T77", op="fwd", B=1, T=77, lens="", H=16, dk=128, dv=128, dtype="bf16", decay="slopes", state=True),
        # the training shape of the benchmark
        dict(name="fwd_train_B4_T4096", op="fwd", B=4, T=4096, lens="", H=16, dk=128, dv=128, dtype="bf16", decay="slopes", state=True),
        # one long document
        dict(name="fwd_long_T65536", op="fwd", B=1, T=65536, lens="", H=32, dk=128, dv=128, dtype="bf16", decay="slopes", state=False),
        # 16 packed prompts of 1,024 to 16,384 tokens, 146,641 in all
        dict(name="fwd_packed_16", op="fwd", B=1, T=146641, lens="benchmark", H=32, dk=128, dv=128, dtype="bf16", decay="slopes", state=True),
        # fp32 inputs, keys of 64 channels
        dict(name="fwd_f32_B4_T1021", op="fwd", B=4, T=1021, lens="", H=16, dk=64, dv=128, dtype="f32", decay="slopes", state=True),
        # the gradients on the training shape
        dict(name="bwd_train_B4_T4096", op="bwd", B=4, T=4096, lens="", H=16, dk=128, dv=128, dtype="bf16", decay="slopes", state=True),
        # gradients of a small packed batch with an empty sequence and one of one token, no decay
        dict(name="bwd_packed_small", op="bwd", B=1, T=1667, lens="1000,0,1,538,128", H=6, dk=64, dv=128, dtype="bf16", decay="none", state=True),
        # one token for each of 256 sequences (the decoding shape of the benchmark) and for one
        dict(name="step_B256_H32", op="step", B=256, H=32, dk=128, dv=128, dtype="bf16", decay="slopes"),
        dict(name="step_B1_H16", op="step", B=1, H=16, dk=128, dv=128, dtype="bf16", decay="slopes"),
        # queries and keys of the packed prompts, RMS norm with weights, rotation of all channels
        dict(name="norm_prompt_T65536", op="norm", B=1, T=65536, Hq=32, Hk=8, d=128, rot=128, dtype="bf16", norm="rms", weights=True, interleaved=False),
        # one token for each of 64 sequences at far positions
        dict(name="norm_step_B64", op="norm", B=64, T=1, Hq=32, Hk=8, d=128, rot=64, dtype="bf16", norm="rms", weights=True, interleaved=False),
        # the gradients on the training shape, RMS norm with weights and rotation
        dict(name="norm_bwd_B4_T4096", op="norm_bwd", B=4, T=4096, Hq=16, Hk=16, d=128, rot=128, dtype="bf16", norm="rms", weights=True, interleaved=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "step", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("fwd", "bwd"):
        H = rng.choice([1, 2, 3, 5, 8, 16, 24, 32])
        T = _log_int(rng, 1, 20000 if op == "fwd" else 8000)
        if dtype == "f32":
            T = max(1, T // 4)
        c = dict(op=op, B=1, T=T, lens="", H=H, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), dtype=dtype,
                 decay=rng.choice(["slopes", "slopes", "strong", "none"]), state=rng.random() < 0.6)
        if rng.random() < 0.5:
            cuts = sorted(rng.randint(0, T) for _ in range(rng.randint(0, 6)))
            c["lens"] = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))
        else:
            c["B"] = rng.choice([1, 1, 2, 3, 4]) if T < 5000 else 1
        return c
    if op == "step":
        return dict(op=op, B=_log_int(rng, 1, 200), H=rng.choice([1, 3, 8, 16, 32]), dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                    dtype=dtype, decay=rng.choice(["slopes", "strong", "none"]))
    d = rng.choice([64, 128, 128, 80, 96, 192, 256])
    Hk = rng.choice([1, 2, 4, 8])
    return dict(op=op, B=rng.choice([1, 2, 5]), T=_log_int(rng, 1, 6000), Hq=Hk * rng.choice([1, 2, 4]), Hk=Hk, d=d,
                rot=rng.choice([0, 32, d // 16 * 16]), dtype=dtype, norm=rng.choice(["rms", "l2"]), weights=rng.random() < 0.6,
                interleaved=rng.random() < 0.4)


# ----------------------------------------------------------------- inputs --
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    if not case["lens"]:
        return [case["T"]] * case["B"]
    if case["lens"] == "benchmark":   # the packed benchmark's 16 lengths, drawn from seed 4
        g = torch.Generator().manual_seed(4)
        return [int(x) for x in torch.randint(1024, 16384 + 1, (16,), generator=g)]
    return [int(x) for x in case["lens"].split(",")]


def _log_decay(kind, H):
    """None, or fixed slopes as such models take them: 2^(-8 (h + 1) / H) per head, fastest first; "strong" is up to 20 times that."""
    if kind == "none":
        return None
    slope = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")
    return -slope * (20.0 if kind == "strong" else 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    op = case["op"]
    if op in ("fwd", "bwd"):
        B, T, H, dk, dv = case["B"], case["T"], case["H"], case["dk"], case["dv"]
        lens = _lens(case)
        s = dict(op=op, lens=lens, q=unit(B, T, H, dk), k=unit(B, T, H, dk), v=normal(B, T, H, dv).to(dt),
                 log_decay=_log_decay(case["decay"], H), S0=None, cu=None)
        if case["lens"]:
            s["cu"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        if case["state"]:
            s["S0"] = 0.1 * normal(len(lens), H, dk, dv)
        if op == "bwd":
            s["d_o"] = normal(B, T, H, dv).to(dt)
            s["dS"] = 0.1 * normal(len(lens), H, dk, dv) if case["state"] else None
        return s
    if op == "step":
        B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
        return dict(op=op, q=unit(B, H, dk), k=unit(B, H, dk), v=normal(B, H, dv).to(dt),
                    log_decay=_log_decay(case["decay"], H), S=0.5 * normal(B, H, dk, dv))
    B, T, Hq, Hk, d, rot = case["B"], case["T"], case["Hq"], case["Hk"], case["d"], case["rot"]
    # queries, keys and values come out of one projection, side by side
    qkv = (normal(B, T, Hq + 2 * Hk, d) * (0.5 + torch.rand(d, generator=g, device="cuda"))).to(dt)
    s = dict(op=op, q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hk], norm=case["norm"], eps=1e-6, interleaved=case["interleaved"],
             wq=None, wk=None, freq=None, pos=None)
    if case["weights"]:
        s["wq"], s["wk"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
    if rot:
        s["freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
        first = torch.randint(0, 100000, (B, 1), generator=g, device="cuda", dtype=torch.int32)
        s["pos"] = first + torch.arange(T, dtype=torch.int32, device="cuda")
    if op == "norm_bwd":
        s["dq"], s["dk"] = normal(B, T, Hq, d).to(dt), normal(B, T, Hk, d).to(dt)
    return s


# -------------------------------------------------------------------- run --
def run(state):
    s = state
    if own:
        from gated_delta_rule_108_b200 import kda
        if s["op"] == "fwd":
            return kda.linear_chunk_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["S0"], cu_seqlens=s["cu"])
        if s["op"] == "bwd":
            r = kda.linear_chunk_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["d_o"], s["S0"], s["dS"], cu_seqlens=s["cu"])
            return r["dq"], r["dk"], r["dv"], r["dS0"]
        if s["op"] == "step":
            return kda.linear_recurrent_step(s["q"], s["k"], s["v"], s["log_decay"], s["S"]), s["S"]
        more = dict(q_weight=s["wq"], k_weight=s["wk"], inv_freq=s["freq"], positions=s["pos"], norm=s["norm"], eps=s["eps"],
                    interleaved=s["interleaved"])
        if s["op"] == "norm":
            return kda.qk_norm_rope(s["q"], s["k"], **more)
        r = kda.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], **more)
        return r["dq"], r["dk"], r["dq_weight"], r["dk_weight"]
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[s["op"]](s)


def _pow(log_decay, n, H):
    """e^(l n) per head in front of n's dimensions, from 64-bit exponents; 1 without a decay."""
    l = torch.zeros(H, dtype=torch.float64, device=n.device) if log_decay is None else log_decay.double()
    return torch.exp(l.view(-1, *[1] * n.dim()) * n.double()).float()


class _Blocks:
    """The tokens of all sequences in blocks of CHUNK that do not cross a sequence's end."""

    def __init__(self, s):
        q, lens = s["q"], torch.tensor(s["lens"])
        dev, N = q.device, len(s["lens"])
        self.N, self.T, self.H = N, q.shape[0] * q.shape[1], q.shape[2]
        count = (lens + CHUNK - 1) // CHUNK
        self.nc = int(count.sum())
        lens, count = lens.to(dev), count.to(dev)
        begin = lens.cumsum(0) - lens            # first token and first block of each sequence
        first = count.cumsum(0) - count
        self.lens = lens
        self.seq = torch.repeat_interleave(torch.arange(N, device=dev), count, output_size=self.nc)
        self.start = (torch.arange(self.nc, device=dev) - first[self.seq]) * CHUNK       # within its sequence
        self.len = torch.minimum(lens[self.seq] - self.start, torch.tensor(CHUNK, device=dev))
        self.end = self.start + self.len
        i = torch.arange(CHUNK, device=dev)
        self.inside = i < self.len[:, None]
        self.at = ((begin[self.seq] + self.start)[:, None] + i).clamp(max=max(self.T - 1, 0))
        t = torch.arange(self.T, device=dev)
        of = torch.searchsorted(lens.cumsum(0), t, right=True)
        self.back = (first[of] + (t - begin[of]) // CHUNK) * CHUNK + (t - begin[of]) % CHUNK
        self.i = i

    def cut(self, x):          # [B, T, H, d] -> fp32 [H, blocks, CHUNK, d], zeros past a block's end
        x = x.reshape(self.T, self.H, -1)[self.at].float() * self.inside[..., None, None]
        return x.permute(2, 0, 1, 3)

    def join(self, x, like):   # and back
        return x.permute(1, 2, 0, 3).reshape(self.nc * CHUNK, self.H, -1)[self.back].reshape(like.shape).to(like.dtype)


def _plain_parts(s):
    b = _Blocks(s)
    l, H = s["log_decay"], b.H
    lag = b.i[:, None] - b.i[None, :]
    D = _pow(l, lag.clamp(min=0), H) * (lag >= 0)                             # [H, C, C]
    into = _pow(l, b.i + 1, H)[:, None, :, None]                              # from a block's start to its token i
    left = _pow(l, (b.len[:, None] - 1 - b.i).clamp(min=0), H)[..., None]     # from its token i to its end
    gap = b.start[:, None] - b.end[None, :]                                   # from the end of block c' to the start of c
    near = (b.seq[:, None] == b.seq[None, :]) & (gap >= 0)
    M = _pow(l, gap.clamp(min=0), H) * near                                   # [H, blocks, blocks]
    return b, D[:, None], into, left, M


def _plain_states(s, b, left, M, k, v):
    """The states that enter each block, and each block's own contribution."""
    l, H = s["log_decay"], b.H
    U = (k * left).transpose(-1, -2) @ v                                      # [H, blocks, dk, dv]
    S = (M @ U.flatten(2)).view_as(U)
    if s["S0"] is not None:
        S = S + _pow(l, b.start, H)[..., None, None] * s["S0"].transpose(0, 1)[:, b.seq]
    return S, U


def _plain_fwd(s):
    b, D, into, left, M = _plain_parts(s)
    q, k, v = b.cut(s["q"]), b.cut(s["k"]), b.cut(s["v"])
    S, U = _plain_states(s, b, left, M, k, v)
    o = q.shape[-1] ** -0.5 * (((q @ k.transpose(-1, -2)) * D) @ v + into * (q @ S))
    to_end = _pow(s["log_decay"], (b.lens[:, None] - b.end).clamp(min=0), b.H) * (torch.arange(b.N, device=q.device)[:, None] == b.seq)
    final = (to_end @ U.flatten(2)).view(b.H, b.N, *U.shape[2:])
    if s["S0"] is not None:
        final = final + _pow(s["log_decay"], b.lens, b.H)[..., None, None] * s["S0"].transpose(0, 1)
    return b.join(o, s["v"]), final.transpose(0, 1).contiguous()


def _plain_bwd(s):
    b, D, into, left, M = _plain_parts(s)
    l, H = s["log_decay"], b.H
    q, k, v, do = b.cut(s["q"]), b.cut(s["k"]), b.cut(s["v"]), b.cut(s["d_o"])
    c = q.shape[-1] ** -0.5
    S, _ = _plain_states(s, b, left, M, k, v)
    V = c * (q * into).transpose(-1, -2) @ do                                 # each block's gift to the states before it
    R = (M.transpose(-1, -2) @ V.flatten(2)).view_as(V)
    from_start = _pow(l, b.start, H).unsqueeze(1) * (torch.arange(b.N, device=q.device)[:, None] == b.seq)
    dS0 = (from_start @ V.flatten(2)).view(H, b.N, *V.shape[2:])
    if s["dS"] is not None:
        dS = s["dS"].transpose(0, 1)
        R = R + _pow(l, b.lens[b.seq] - b.end, H)[..., None, None] * dS[:, b.seq]
        dS0 = dS0 + _pow(l, b.lens, H)[..., None, None] * dS
    dP, P = (do @ v.transpose(-1, -2)) * D, (q @ k.transpose(-1, -2)) * D
    dq = c * (dP @ k + into * (do @ S.transpose(-1, -2)))
    dk = c * (dP.transpose(-1, -2) @ q) + left * (v @ R.transpose(-1, -2))
    dv = c * (P.transpose(-1, -2) @ do) + left * (k @ R)
    return b.join(dq, s["q"]), b.join(dk, s["k"]), b.join(dv, s["v"]), dS0.transpose(0, 1).contiguous()


def _plain_step(s):
    q, k, v, S = s["q"].float(), s["k"].float(), s["v"].float(), s["S"]
    if s["log_decay"] is not None:
        S.mul_(s["log_decay"].exp()[:, None, None])
    S.add_(k[..., None] * v[..., None, :])
    return (q.shape[-1] ** -0.5 * (q[..., None, :] @ S).squeeze(-2)).to(s["v"].dtype), S


def _angles(s, dtype):
    a = s["pos"].double()[..., None, None] * s["freq"].double()               # [B, T, 1, rot / 2]
    return a.cos().to(dtype), a.sin().to(dtype)


def _turn(s, x, cos, sin):
    """The first 2 len(freq) channels of x in pairs, turned."""
    h = s["freq"].numel()
    r, rest = x[..., :2 * h], x[..., 2 * h:]
    a, b = (r[..., 0::2], r[..., 1::2]) if s["interleaved"] else (r[..., :h], r[..., h:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _scale_of(s, x):
    m = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((m / x.shape[-1] if s["norm"] == "rms" else m) + s["eps"])


def _plain_norm_of(s, x, w, turn):
    x = x.float()
    n = x * _scale_of(s, x)
    n = n if w is None else n * w
    return n if turn is None else _turn(s, n, *turn)


def _plain_norm(s):
    turn = None if s["freq"] is None else _angles(s, torch.float32)
    return _plain_norm_of(s, s["q"], s["wq"], turn).to(s["q"].dtype), _plain_norm_of(s, s["k"], s["wk"], turn).to(s["k"].dtype)


def _plain_norm_bwd_of(s, x, w, dy, turn):
    dt, x, dn = x.dtype, x.float(), dy.float()
    if turn is not None:
        dn = _turn(s, dn, turn[0], -turn[1])
    r = _scale_of(s, x)
    dw = None if w is None else (dn * x * r).sum((0, 1, 2))
    dn = dn if w is None else dn * w
    m = (dn * x).sum(-1, keepdim=True)
    m = m / x.shape[-1] if s["norm"] == "rms" else m
    return (r * dn - r ** 3 * m * x).to(dt), dw


def _plain_norm_bwd(s):
    turn = None if s["freq"] is None else _angles(s, torch.float32)
    dq, dwq = _plain_norm_bwd_of(s, s["q"], s["wq"], s["dq"], turn)
    dk, dwk = _plain_norm_bwd_of(s, s["k"], s["wk"], s["dk"], turn)
    return dq, dk, dwq, dwk


# ------------------------------------------------------------------- work --
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("fwd", "bwd"):
        n, N, H, dk, dv = case["B"] * case["T"], len(_lens(case)), case["H"], case["dk"], case["dv"]
        one = N * H * dk * dv * 4   # the states of all sequences
        if op == "fwd":             # q, k, v read, o written; the states; each token is added to a state and read from it
            return {"bytes": n * H * (2 * dk + 2 * dv) * e + one * (1 + case["state"]), "flops": 4 * n * H * dk * dv}
        # q, k, v, d_o read, dq, dk, dv written; both states built, dq, dk and dv read from them
        return {"bytes": n * H * (4 * dk + 3 * dv) * e + one * (1 + 2 * case["state"]), "flops": 10 * n * H * dk * dv}
    if op == "step":
        n, dk, dv = case["B"] * case["H"], case["dk"], case["dv"]
        return {"bytes": n * (2 * dk * dv * 4 + (2 * dk + 2 * dv) * e), "flops": 4 * n * dk * dv}
    n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
    more = case["B"] * case["T"] * 4 * (case["rot"] > 0) + case["d"] * 8 * case["weights"]
    return {"bytes": n * e * (2 if op == "norm" else 3) + more, "flops": n * (6 if op == "norm" else 16)}


# ------------------------------------------------------------------ exact --
def _exact_of(a, b, c, l, first, shift):
    """sum_i [i <= r] e^(l (r - i)) <a_r, b_i> c_i + e^(l (r + shift)) a_r first, in fp64, a block of rows at a time."""
    T, R = a.shape[0], 2048
    powers = torch.exp(l * torch.arange(T + 1, dtype=torch.float64, device=a.device))
    out = torch.zeros(T, c.shape[1], dtype=torch.float64, device=a.device)
    lags = torch.cat((torch.zeros(R, dtype=torch.float64, device=a.device), powers))   # lags[R + m] = e^(l m), 0 for m < 0
    for r0 in range(0, T, R):
        n = min(R, T - r0)
        # keys from the last to the first: column y is key r0 + n - 1 - y, so the lag of row r0 + x is x + y - n + 1
        D = lags.as_strided((n, r0 + n), (1, 1), R - n + 1)
        out[r0:r0 + n] = ((a[r0:r0 + n] @ b[:r0 + n].flip(0).T) * D) @ c[:r0 + n].flip(0)
    if first is not None:
        steps = torch.arange(T, dtype=torch.float64, device=a.device) + shift
        out += torch.exp(l * steps)[:, None] * (a @ first)
    return out


def _exact_linear(s, case):
    lens, H = s["lens"], case["H"]
    flat = {n: s[n].reshape(-1, H, s[n].shape[-1]) for n in ("q", "k", "v", "d_o") if n in s}
    bwd = s["op"] == "bwd"
    names = ("q", "k", "v") if bwd else ("v",)
    outs = [torch.zeros(flat[n].shape, dtype=torch.float64, device="cuda") for n in names]
    states = torch.zeros(len(lens), H, case["dk"], case["dv"], dtype=torch.float64, device="cuda")
    scale, t = case["dk"] ** -0.5, 0
    for n, L in enumerate(lens):
        for h in range(H):
            l = 0.0 if s["log_decay"] is None else float(s["log_decay"][h])
            x = {m: y[t:t + L, h].double() for m, y in flat.items()}
            S0 = None if s["S0"] is None else s["S0"][n, h].double()
            i = torch.arange(L, dtype=torch.float64, device="cuda")
            if not bwd:
                outs[0][t:t + L, h] = scale * _exact_of(x["q"], x["k"], x["v"], l, S0, 1)
                states[n, h] = (x["k"] * torch.exp(l * (L - 1 - i))[:, None]).T @ x["v"]
                if S0 is not None:
                    states[n, h] += math.exp(l * L) * S0
                continue
            dS = None if s["dS"] is None else s["dS"][n, h].double() / scale
            back = {m: y.flip(0) for m, y in x.items()}   # the adjoint runs from the last token to the first
            outs[0][t:t + L, h] = scale * _exact_of(x["d_o"], x["v"], x["k"], l, None if S0 is None else S0.T, 1)
            outs[1][t:t + L, h] = scale * _exact_of(back["v"], back["d_o"], back["q"], l, None if dS is None else dS.T, 0).flip(0)
            outs[2][t:t + L, h] = scale * _exact_of(back["k"], back["q"], back["d_o"], l, dS, 0).flip(0)
            states[n, h] = scale * (x["q"] * torch.exp(l * (i + 1))[:, None]).T @ x["d_o"]
            if dS is not None:
                states[n, h] += math.exp(l * L) * scale * dS
        t += L
    outs = [o.reshape(s[n].shape) for o, n in zip(outs, names)]
    return (*outs, states)


def _exact_rows(s, x, w, dy):
    """One query or key tensor in fp64: the outputs, or (dy given) the gradients by the Jacobian written as matrices of the row."""
    d = x.shape[-1]
    x = x.double()
    m = x.square().sum(-1, keepdim=True)
    r = 1 / ((m / d if s["norm"] == "rms" else m) + s["eps"]).sqrt()
    w64 = torch.ones(d, dtype=torch.float64, device="cuda") if w is None else w.double()
    if s["freq"] is not None:
        h = s["freq"].numel()
        j = torch.arange(h, device="cuda")
        at = torch.stack((2 * j, 2 * j + 1) if s["interleaved"] else (j, j + h))      # [2, h] channels of each pair
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["pos"].double()[..., None, None] * s["freq"].double())

    def turned(y, by):
        z = torch.complex(y[..., at[0]], y[..., at[1]]) * by
        y = y.clone()
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
        return y

    if dy is None:
        y = x * r * w64
        return y if s["freq"] is None else turned(y, turn)
    g = dy.double()
    if s["freq"] is not None:
        g = turned(g, turn.conj())
    unit = x * r
    dw = None if w is None else (g * unit).flatten(0, 2).sum(0)
    g = g * w64
    along = (g * unit).sum(-1, keepdim=True) / (d if s["norm"] == "rms" else 1)
    return (g - unit * along) * r, dw


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("fwd", "bwd"):
        return _exact_linear(s, case)
    if s["op"] == "step":
        a = 1.0 if s["log_decay"] is None else s["log_decay"].double().exp()[:, None, None]
        S = a * s["S"].double() + torch.einsum("bhi,bhj->bhij", s["k"].double(), s["v"].double())
        return case["dk"] ** -0.5 * torch.einsum("bhi,bhij->bhj", s["q"].double(), S), S
    if s["op"] == "norm":
        return _exact_rows(s, s["q"], s["wq"], None), _exact_rows(s, s["k"], s["wk"], None)
    (dq, dwq), (dk, dwk) = _exact_rows(s, s["q"], s["wq"], s["dq"]), _exact_rows(s, s["k"], s["wk"], s["dk"])
    return dq, dk, dwq, dwk
