"""What a linear-attention layer runs besides its projections, case by case: the
queries' and keys' norm with the rotation (``rope``), linear attention with a decay
for each head (``la``), and the gated norm of its output (``gated``).

``run`` computes a case in plain 32-bit torch operations, or, where ``own`` is
true, with the framework's operators; ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one user's next token: a single sequence, six heads; nothing but latency
        dict(name="la_step_B1_H6", op="la_decode", B=1, T=1, H=6, K=128, V=128, dtype="bf16", decay="slopes"),
        # a serving batch's next tokens: 256 sequences with warm states (268 MB of state)
        dict(name="la_step_B256_H16", op="la_decode", B=256, T=1, H=16, K=128, V=128, dtype="bf16", decay="slopes"),
        # one prompt of an odd length, v taken out of a fused projection
        dict(name="la_prompt_T777_H16", op="la_fwd", B=1, T=777, H=16, K=128, V=128, dtype="bf16", decay="slopes", fused=True),
        # a long document read in one call, the state kept for what follows
        dict(name="la_stream_T32768_H16", op="la_fwd", B=1, T=32768, H=16, K=128, V=128, dtype="bf16", decay="slopes"),
        # a training step's layer at the repository's training shape
        dict(name="la_train_B8_T4096_H6", op="la_train", B=8, T=4096, H=6, K=128, V=128, dtype="bf16", decay="slopes"),
        # training on ragged batches of a smaller model: odd length, unequal widths, heads that hardly forget
        dict(name="la_train_B3_T1537_K64_V128", op="la_train", B=3, T=1537, H=5, K=64, V=128, dtype="bf16", decay="slow"),
        # a unit-test sized training step in 32 bits
        dict(name="la_train_f32_T64_K16", op="la_train", B=1, T=64, H=2, K=16, V=16, dtype="f32", decay="slopes"),
        # fine-tuning in 32 bits, no decay in any head
        dict(name="la_train_f32_B2_T1024_K64", op="la_train", B=2, T=1024, H=4, K=64, V=64, dtype="f32", decay="none"),
        # the next token's queries and keys of a small serving batch, each at a position of its own
        dict(name="rope_step_B8_H16", op="rope_fwd", B=8, T=1, H=16, Hk=16, D=128, R=128, dtype="bf16", interleaved=False, fused=False),
        # queries and keys of a training step, taken out of a fused projection, forward and backward
        dict(name="rope_train_B8_T4096_H6", op="rope_train", B=8, T=4096, H=6, Hk=6, D=128, R=128, dtype="bf16", interleaved=False, fused=True),
        # the output norm of a serving batch's next tokens
        dict(name="gated_step_B256_H16", op="gated_fwd", B=256, T=1, H=16, D=128, dtype="bf16", fused=False),
        # the output norm of a training step, forward and backward
        dict(name="gated_train_B8_T4096_H6", op="gated_train", B=8, T=4096, H=6, D=128, dtype="bf16", fused=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["la_decode", "la_fwd", "la_fwd", "la_train", "la_train", "la_train", "rope_fwd", "rope_train", "gated_fwd", "gated_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    H = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
    if op == "la_decode":
        return dict(op=op, B=_log(rng, 1, 4096 // H), T=1, H=H, K=rng.choice([16, 32, 64, 128]), V=rng.choice([16, 32, 64, 128]), dtype=dtype,
                    decay=rng.choice(["slopes", "slow", "none"]))
    if op in ("la_fwd", "la_train"):
        # most of the range is what trains and serves: wide heads, many tokens
        most = (196608 if op == "la_train" else 524288) // (1 if dtype == "bf16" else 4)
        T = _log(rng, 1, min(32768, most // H))
        return dict(op=op, B=_log(rng, 1, max(1, min(64, most // (H * T)))), T=T, H=H, K=rng.choice([16, 32, 64, 128, 128]), V=rng.choice([16, 32, 64, 128, 128]),
                    dtype=dtype, decay=rng.choice(["slopes", "slow", "none"]), fused=rng.random() < 0.3)
    T = _log(rng, 1, 8192)
    B = _log(rng, 1, max(1, min(256, 196608 // (H * T))))
    D = rng.choice([32, 64, 96, 128, 128, 256])
    if op in ("rope_fwd", "rope_train"):
        return dict(op=op, B=B, T=T, H=H, Hk=rng.choice([n for n in range(1, H + 1) if H % n == 0]), D=D, R=rng.choice([D, D, D // 2]), dtype=dtype,
                    interleaved=rng.random() < 0.3, fused=rng.random() < 0.5)
    return dict(op=op, B=B, T=T, H=H, D=D, dtype=dtype, fused=rng.random() < 0.5)


def _log_decay(kind, H, device):
    h = torch.arange(1, H + 1, dtype=torch.float32, device=device)
    if kind == "slopes":  # a geometric ladder of memory lengths, a few tokens to a few hundred
        return -torch.exp2(-8.0 * h / H)
    if kind == "slow":  # memories of about 100 to 4000 tokens
        return torch.log1p(-torch.exp2(-7.0 - 5.0 * h / H))
    return torch.zeros(H, dtype=torch.float32, device=device)


def prepare(case, seed):
    dev = torch.device("cuda")
    rng = torch.Generator(device=dev)
    rng.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    B, T, H = case["B"], case["T"], case["H"]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=rng, device=dev) * std).to(dtype)

    def heads(n, width):  # rows of their own, or a slice of a fused projection's
        if case.get("fused"):
            return normal(B, T, 2 * n * width + 64)[..., 64:64 + n * width].unflatten(-1, (n, width))
        return normal(B, T, n, width)

    s = dict(case=case)
    if case["op"].startswith("la_"):
        K, V = case["K"], case["V"]
        # rows as the q, k norm leaves them, the query's scale in its weight
        s["q"] = normal(B, T, H, K, std=K ** -0.5)
        s["k"] = normal(B, T, H, K)
        s["v"] = heads(H, V)
        s["log_decay"] = _log_decay(case["decay"], H, dev)
        s["state"] = normal(B, H, V, K, dtype=torch.float32, std=0.5)
        if case["op"] == "la_train":
            s["d_o"] = normal(B, T, H, V)
            s["d_final"] = normal(B, H, V, K, dtype=torch.float32, std=0.01)
    elif case["op"].startswith("rope_"):
        D, R, Hk = case["D"], case["R"], case["Hk"]
        s["q"], s["k"] = heads(H, D), heads(Hk, D)
        s["wq"] = (1 + 0.1 * torch.randn(D, generator=rng, device=dev)).to(dt)
        s["wk"] = (1 + 0.1 * torch.randn(D, generator=rng, device=dev)).to(dt)
        rows = max(T, 4096)
        freq = 10000.0 ** (-torch.arange(R // 2, device=dev, dtype=torch.float64) * 2 / R)
        angle = torch.arange(rows, device=dev, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        start = torch.randint(0, rows - T + 1, (B, 1), generator=rng, device=dev)
        s["positions"] = (start + torch.arange(T, device=dev)).to(torch.int32)
        if case["op"] == "rope_train":
            s["dq"], s["dk"] = normal(B, T, H, D), normal(B, T, Hk, D)
    else:
        D = case["D"]
        s["x"] = normal(B, T, H, D, std=2.0)
        s["gate"] = heads(H, D)
        s["w"] = (1 + 0.1 * torch.randn(D, generator=rng, device=dev)).to(dt)
        if case["op"] == "gated_train":
            s["dy"] = normal(B, T, H, D)
    return s


# ---------------------------------------------------------------- plain forms

CHUNK = 128


def _powers(g, e):
    """exp(g * e) per head, [H, *e.shape], for exponents e >= 0."""
    return torch.exp(g.view(-1, *([1] * e.dim())) * e)


def _la_scan(a, b, c, g, m0, backward):
    """out_r = sum over s up to r (from r on, where `backward`) of
    gamma^|r-s| (a_r . b_s) c_s, plus the part of the state m0 [B,H,Dc,Db] that
    enters; and the state that leaves."""
    B, T, H, _ = a.shape
    rev = 1 if backward else 0
    if backward:
        a, b, c = a.flip(1), b.flip(1), c.flip(1)
    n = -(-T // CHUNK)
    t = torch.arange(T, device=a.device, dtype=torch.float32)
    cw = c * _powers(g, T - 1 - t + rev).t()[None, :, :, None]
    last = torch.exp(g * T)[None, :, None, None] * m0 + cw.permute(0, 2, 3, 1) @ b.permute(0, 2, 1, 3)
    enter = _powers(g, t + 1 - rev).t()[None, :, :, None] * (a.permute(0, 2, 1, 3) @ m0.transpose(-1, -2)).permute(0, 2, 1, 3)

    def chunks(x):
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * CHUNK - T))
        return x.reshape(B, n, CHUNK, H, -1).permute(0, 3, 1, 2, 4)

    a, b, c = chunks(a), chunks(b), chunks(c)
    i = torch.arange(CHUNK, device=a.device, dtype=torch.float32)
    m = torch.arange(n, device=a.device, dtype=torch.float32)
    near = _powers(g, (i[:, None] - i[None, :]).clamp(min=0)) * (i[:, None] >= i[None, :])
    out = ((a @ b.transpose(-1, -2)) * near[:, None]) @ c
    part = (c * _powers(g, CHUNK - 1 - i)[None, :, None, :, None]).transpose(-1, -2) @ b
    link = _powers(g, (CHUNK * (m[:, None] - 1 - m[None, :])).clamp(min=0)) * (m[:, None] > m[None, :])
    begin = (link @ part.flatten(-2)).view(B, H, n, *part.shape[-2:])
    out = out + _powers(g, i + 1)[None, :, None, :, None] * (a @ begin.transpose(-1, -2))
    out = out.permute(0, 2, 3, 1, 4).reshape(B, n * CHUNK, H, -1)[:, :T] + enter
    return (out.flip(1) if backward else out), last


def _plain_la(s):
    op, dt, g = s["case"]["op"], s["q"].dtype, s["log_decay"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if op == "la_decode":
        state = torch.exp(g)[None, :, None, None] * s["state"] + v[:, 0, :, :, None] * k[:, 0, :, None, :]
        s["state"].copy_(state)
        return {"o": (state @ q[:, 0, :, :, None])[..., 0][:, None].to(dt), "state": s["state"]}
    o, final = _la_scan(q, k, v, g, s["state"], False)
    r = {"o": o.to(dt), "final_state": final}
    if op == "la_train":
        d_o = s["d_o"].float()
        r["dq"] = _la_scan(d_o, v, k, g, s["state"].transpose(-1, -2), False)[0].to(dt)
        r["dk"] = _la_scan(v, d_o, q, g, s["d_final"].transpose(-1, -2), True)[0].to(dt)
        dv, d0 = _la_scan(k, q, d_o, g, s["d_final"], True)
        r["dv"], r["d_initial_state"] = dv.to(dt), d0
    return r


def _rms(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _turn(x, c, s, interleaved):
    """The rotation of the first dimensions of each row by the angle of (c, s)."""
    n = c.shape[-1]
    if interleaved:
        x1, x2 = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack((x1 * c - x2 * s, x2 * c + x1 * s), -1).flatten(-2)
    else:
        x1, x2 = x[..., :n], x[..., n:2 * n]
        y = torch.cat((x1 * c - x2 * s, x2 * c + x1 * s), -1)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _norm_grads(x, w, dn):
    r = _rms(x)
    xh, t = x * r, dn * w
    return r * (t - xh * (t * xh).mean(-1, keepdim=True)), (dn * xh).sum((0, 1, 2))


def _plain_rope(s):
    dt, inter = s["q"].dtype, s["case"]["interleaved"]
    at = s["positions"].long()
    c, n = s["cos"][at][:, :, None], s["sin"][at][:, :, None]
    q, k, wq, wk = s["q"].float(), s["k"].float(), s["wq"].float(), s["wk"].float()
    r = {"q": _turn(q * _rms(q) * wq, c, n, inter).to(dt), "k": _turn(k * _rms(k) * wk, c, n, inter).to(dt)}
    if s["case"]["op"] == "rope_train":
        dq, dwq = _norm_grads(q, wq, _turn(s["dq"].float(), c, -n, inter))
        dk, dwk = _norm_grads(k, wk, _turn(s["dk"].float(), c, -n, inter))
        r.update(dq=dq.to(dt), dk=dk.to(dt), dwq=dwq.to(dt), dwk=dwk.to(dt))
    return r


def _plain_gated(s):
    dt = s["x"].dtype
    x, z, w = s["x"].float(), s["gate"].float(), s["w"].float()
    sig = 1 / (1 + torch.exp(-z))
    act = z * sig
    xw = x * _rms(x) * w
    r = {"y": (xw * act).to(dt)}
    if s["case"]["op"] == "gated_train":
        dy = s["dy"].float()
        dx, dw = _norm_grads(x, w, dy * act)
        r.update(dx=dx.to(dt), dgate=(dy * xw * (sig + act * (1 - sig))).to(dt), dw=dw.to(dt))
    return r


# ------------------------------------------------------- the framework's calls

def _own_la(s):
    from gated_delta_rule_19_gb300 import gdn
    op = s["case"]["op"]
    q, k, v, g = s["q"], s["k"], s["v"], s["log_decay"]
    if op == "la_decode":
        o, state = gdn.gdn_la_decode(q, k, v, g, s["state"])
        return {"o": o, "state": state}
    train = op == "la_train"
    o, final, saved = gdn.gdn_la_fwd(q, k, v, g, s["state"], saved=train)
    r = {"o": o, "final_state": final}
    if train:
        r["dq"], r["dk"], r["dv"], r["d_initial_state"] = gdn.gdn_la_bwd(q, k, v, g, s["state"], s["d_o"], s["d_final"], saved=saved)
    return r


def _own_rope(s):
    from gated_delta_rule_19_gb300 import gdn
    args = (s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"])
    inter = s["case"]["interleaved"]
    r = dict(zip(("q", "k"), gdn.gdn_qk_norm_rope_fwd(*args, eps=EPS, interleaved=inter)))
    if s["case"]["op"] == "rope_train":
        r.update(zip(("dq", "dk", "dwq", "dwk"), gdn.gdn_qk_norm_rope_bwd(*args, s["dq"], s["dk"], eps=EPS, interleaved=inter)))
    return r


def _own_gated(s):
    from gated_delta_rule_19_gb300 import gdn
    r = {"y": gdn.gdn_gated_norm_fwd(s["x"], s["gate"], s["w"], eps=EPS)}
    if s["case"]["op"] == "gated_train":
        r["dx"], r["dgate"], r["dw"] = gdn.gdn_gated_norm_bwd(s["x"], s["gate"], s["w"], s["dy"], eps=EPS)
    return r


def run(state):
    kind = state["case"]["op"].split("_")[0]
    if own:
        return {"la": _own_la, "rope": _own_rope, "gated": _own_gated}[kind](state)
    return {"la": _plain_la, "rope": _plain_rope, "gated": _plain_gated}[kind](state)


# ---------------------------------------------------------- the work of a case

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    rows = case["B"] * case["T"] * case["H"]
    op = case["op"]
    if op.startswith("la_"):
        K, V = case["K"], case["V"]
        state = 4 * case["B"] * case["H"] * K * V
        b = rows * (2 * K + 2 * V) * e + 2 * state + 4 * case["H"]  # q, k, v in, o out, the state in and out
        f = rows * 4 * K * V  # the state's update and its reading
        if op == "la_train":  # q, k, v, d_o and the two end states in, dq, dk, dv and the first state's gradient out
            b += rows * (4 * K + 3 * V) * e + 3 * state + 4 * case["H"]
            f += rows * 10 * K * V  # the state and its gradient, one product for each of dq, dk, dv
        return {"bytes": b, "flops": f}
    D = case["D"]
    if op.startswith("rope_"):
        rows = case["B"] * case["T"] * (case["H"] + case["Hk"])
        table = case["B"] * case["T"] * (case["R"] * 4 + 4)  # a cosine and a sine for each pair, and the position
        b, f = rows * 2 * D * e + table + 2 * D * e, rows * (4 * D + 3 * case["R"])
        if op == "rope_train":
            b, f = b + rows * 3 * D * e + table + 4 * D * e, f + rows * (10 * D + 3 * case["R"])
        return {"bytes": b, "flops": f}
    b, f = rows * 3 * D * e + D * e, rows * 9 * D
    if op == "gated_train":
        b, f = b + rows * 5 * D * e + 2 * D * e, f + rows * 20 * D
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------- in 64 bits

def _exact_la(q, k, v, g, state, step=64):
    """The recurrence S <- gamma S + v k^T, o = S q, `step` tokens at a time."""
    gamma = torch.exp(g)
    outs = []
    for t0 in range(0, q.shape[1], step):
        qc, kc, vc = (x[:, t0:t0 + step].transpose(1, 2) for x in (q, k, v))
        n = qc.shape[2]
        e = torch.arange(n, device=q.device, dtype=torch.float64)
        dist = e[:, None] - e[None, :]
        keep = torch.where(dist >= 0, gamma[:, None, None] ** dist.clamp(min=0), torch.zeros((), dtype=torch.float64, device=q.device))
        score = torch.einsum("bhrk,bhsk->bhrs", qc, kc) * keep
        before = torch.einsum("bhrk,bhvk->bhrv", qc, state) * (gamma[:, None] ** (e + 1))[None, :, :, None]
        outs.append((before + torch.einsum("bhrs,bhsv->bhrv", score, vc)).transpose(1, 2))
        fade = (gamma[:, None] ** (n - 1 - e))[None, :, :, None]
        state = state * (gamma ** n)[None, :, None, None] + torch.einsum("bhsv,bhsk->bhvk", vc * fade, kc)
    return torch.cat(outs, 1), state


def _exact_rows(x, w, cos=None, sin=None, interleaved=False):
    y = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w
    if cos is None:
        return y
    n = cos.shape[-1]
    turned = y[..., :2 * n]
    pairs = turned.unflatten(-1, (n, 2)) if interleaved else turned.unflatten(-1, (2, n)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * torch.complex(cos, sin)
    z = torch.view_as_real(z)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, y[..., 2 * n:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    train = case["op"].endswith("_train")
    d = {n: t.double().requires_grad_(train) for n, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point()}
    with torch.set_grad_enabled(train):
        if case["op"].startswith("la_"):
            o, final = _exact_la(d["q"], d["k"], d["v"], d["log_decay"].detach(), d["state"])
            if case["op"] == "la_decode":
                return {"o": o, "state": final}
            r = {"o": o, "final_state": final}
            if train:
                r.update(zip(("dq", "dk", "dv", "d_initial_state"),
                             torch.autograd.grad((o, final), (d["q"], d["k"], d["v"], d["state"]), (d["d_o"], d["d_final"]))))
        elif case["op"].startswith("rope_"):
            at = s["positions"].long()
            c, n = d["cos"].detach()[at][:, :, None], d["sin"].detach()[at][:, :, None]
            q = _exact_rows(d["q"], d["wq"], c, n, case["interleaved"])
            k = _exact_rows(d["k"], d["wk"], c, n, case["interleaved"])
            r = {"q": q, "k": k}
            if train:
                r.update(zip(("dq", "dk", "dwq", "dwk"), torch.autograd.grad((q, k), (d["q"], d["k"], d["wq"], d["wk"]), (d["dq"], d["dk"]))))
        else:
            y = _exact_rows(d["x"], d["w"]) * d["gate"] * torch.sigmoid(d["gate"])
            r = {"y": y}
            if train:
                r.update(zip(("dx", "dgate", "dw"), torch.autograd.grad(y, (d["x"], d["gate"], d["w"]), d["dy"])))
    return {n: t.detach() for n, t in r.items()}
