"""Plain fp64 forms for the tests of the linear attention with one decay per head
and of the query/key norm with rotation: the definitions, token by token and row by
row, and bounds on what rounding may do to the kernels' results."""
import torch


def lens_of(B, T, cu):
    return [T] * B if cu is None else [int(b - a) for a, b in zip(cu[:-1], cu[1:])]


def forward(q, k, v, log_decay, S0=None, cu=None):
    """o and the final states in fp64, and the same with every product taken in
    magnitude (what rounding errors scale with)."""
    B, T, H, dk = q.shape
    dv, lens = v.shape[-1], lens_of(B, T, cu)
    q, k, v = (x.double().reshape(B * T, H, -1) for x in (q, k, v))
    a = torch.ones(H, dtype=torch.float64) if log_decay is None else log_decay.double().exp()
    o, om = torch.zeros(B * T, H, dv, dtype=torch.float64), torch.zeros(B * T, H, dv, dtype=torch.float64)
    Sf, Sm = (torch.zeros(len(lens), H, dk, dv, dtype=torch.float64) for _ in range(2))
    t = 0
    for n, L in enumerate(lens):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if S0 is None else S0[n].double()
        M = S.abs()
        for _ in range(L):
            kv = k[t][:, :, None] * v[t][:, None, :]
            S, M = a[:, None, None] * S + kv, a[:, None, None] * M + kv.abs()
            o[t] = dk ** -0.5 * (q[t][:, None, :] @ S)[:, 0]
            om[t] = dk ** -0.5 * (q[t].abs()[:, None, :] @ M)[:, 0]
            t += 1
        Sf[n], Sm[n] = S, M
    return o.reshape(B, T, H, dv), Sf, om.reshape(B, T, H, dv), Sm


def backward(q, k, v, log_decay, d_o, S0=None, dS=None, cu=None):
    """dq, dk, dv, dS0 in fp64 by the adjoint recurrence, and their magnitudes."""
    B, T, H, dk = q.shape
    dv, lens = v.shape[-1], lens_of(B, T, cu)
    q, k, v, d_o = (x.double().reshape(B * T, H, -1) for x in (q, k, v, d_o))
    a = torch.ones(H, dtype=torch.float64) if log_decay is None else log_decay.double().exp()
    c = dk ** -0.5
    g = {n: torch.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    m = {n: torch.zeros_like(x) for n, x in g.items()}
    g["dS0"], m["dS0"] = (torch.zeros(len(lens), H, dk, dv, dtype=torch.float64) for _ in range(2))

    def row(S, x):     # S x per head
        return (S @ x[:, :, None])[..., 0]

    t = 0
    for n, L in enumerate(lens):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if S0 is None else S0[n].double()
        M = S.abs()
        for i in range(t, t + L):
            kv = k[i][:, :, None] * v[i][:, None, :]
            S, M = a[:, None, None] * S + kv, a[:, None, None] * M + kv.abs()
            g["dq"][i], m["dq"][i] = c * row(S, d_o[i]), c * row(M, d_o[i].abs())
        G = torch.zeros(H, dk, dv, dtype=torch.float64) if dS is None else dS[n].double()
        N = G.abs()
        for i in range(t + L - 1, t - 1, -1):
            qd = c * q[i][:, :, None] * d_o[i][:, None, :]
            G, N = G + qd, N + qd.abs()
            g["dk"][i], m["dk"][i] = row(G, v[i]), row(N, v[i].abs())
            g["dv"][i], m["dv"][i] = row(G.transpose(1, 2), k[i]), row(N.transpose(1, 2), k[i].abs())
            G, N = a[:, None, None] * G, a[:, None, None] * N
        g["dS0"][n], m["dS0"][n] = G, N
        t += L
    for d in (g, m):
        for n in ("dq", "dk", "dv"):
            d[n] = d[n].reshape(B, T, H, -1)
    return g, m


def assert_close(x, ref, mag, dtype, what, tokens, state=False):
    """|x - ref| against what roundings allow, element by element, and in 2-norm.

    Sums of n terms in fp32 are off by at most n 2^-24 of the terms' magnitudes
    `mag`; chunks of 128 tokens and dk <= 128 channels give n <= 300 per chunk, and
    errors of earlier chunks come on top: (300 + 24 chunks) 2^-24, doubled for the
    tensor core's own truncating adds.  The exponentials and weights add 2^-22.
    bf16 inputs: the operand Z is rounded once (2^-8 of mag) and P and the weighted
    c in two parts (2^-16 each); the result once more (2^-8 of its value).  States
    have three parts (2^-24).  In 2-norm a rounding is a uniform error of 2^-8 /
    sqrt(3), and two of them stay below 2^-8: 4e-3.
    """
    x, ref, mag = x.double().cpu(), ref.double(), mag.double()
    assert x.shape == ref.shape, what
    chunks = -(-tokens // 128)
    n = 2 * (300 + 24 * chunks) * 2.0 ** -24 + 2.0 ** -22
    tol = n * mag + 1e-30
    if dtype == torch.bfloat16 and not state:
        tol = tol + 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -15) * mag
    bad = ~((x - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, first at {bad.nonzero()[0].tolist()}"
    if dtype == torch.bfloat16 and not state and ref.norm() > 0:
        rel = float((x - ref).norm() / ref.norm())
        assert rel <= 4e-3, f"{what}: relative error {rel:.2e}"


def rotate(y, pos, freq, interleaved, back=False):
    h = freq.numel()
    if h == 0:
        return y
    t = pos.double()[..., None, None] * freq.double()
    c, s = t.cos(), t.sin() * (-1 if back else 1)
    a, b = (y[..., 0:2 * h:2], y[..., 1:2 * h:2]) if interleaved else (y[..., :h], y[..., h:2 * h])
    out = y.clone()
    if interleaved:
        out[..., 0:2 * h:2], out[..., 1:2 * h:2] = a * c - b * s, b * c + a * s
    else:
        out[..., :h], out[..., h:2 * h] = a * c - b * s, b * c + a * s
    return out


def norm_rope(x, w, freq, pos, norm, eps, interleaved):
    """One of queries or keys, [B, T, H, d] -> fp64."""
    x = x.double()
    m = x.square().sum(-1, keepdim=True)
    n = x / ((m / x.shape[-1] if norm == "rms" else m) + eps).sqrt()
    n = n if w is None else n * w.double()
    return n if freq is None else rotate(n, pos, freq, interleaved)
