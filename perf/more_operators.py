"""What surrounds a linear-attention layer in its block, case by case: the residual's
addition with the RMS norm, also with an 8-bit output (``norm``, ``quant``); the queries'
and keys' norm with a rotation by several positions (``axes``); the gradients' global norm
and clipping (``clip``); and the states of waiting sequences, parked in 8 bits and resumed
(``swap``).

``run`` computes a case in plain 32-bit torch operations, or, where ``own`` is
true, with the framework's operators; ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
MOST = 448.0        # e4m3's largest number
LEAST = 2.0 ** -126  # the least scale, float32's smallest normal number


def listed():
    return [
        # the next tokens of eight sequences in front of a layer of 16 heads of 128
        dict(name="norm_step_B8_D2048", op="norm_fwd", B=8, T=1, D=2048, dtype="bf16", residual="bf16", fused=False),
        # the norm of a training step at the repository's training shape (6 heads of 128)
        dict(name="norm_train_B8_T4096_D768", op="norm_train", B=8, T=4096, D=768, dtype="bf16", residual="bf16", fused=False),
        # training with a residual stream in 32 bits: odd lengths and width, x a slice of a wider row
        dict(name="norm_train_B3_T1537_D1000_r32", op="norm_train", B=3, T=1537, D=1000, dtype="bf16", residual="f32", fused=True),
        # a serving batch's next tokens, for a projection in 8 bits with a scale for each row
        dict(name="quant_step_B256_D2048", op="quant", B=256, T=1, D=2048, dtype="bf16", residual="bf16", fused=False, group=0),
        # prompts of a wide model, with a scale for each 128 columns
        dict(name="quant_prompt_T7777_D4096", op="quant", B=1, T=7777, D=4096, dtype="bf16", residual="bf16", fused=False, group=128),
        # next tokens of a serving batch of a model that reads images: text, its three positions alike
        dict(name="axes_step_B8_H16", op="axes_fwd", B=8, T=1, H=16, Hk=16, D=128, R=128, dtype="bf16", kind="blocks", interleaved=False, fused=False),
        # a training step on video between text, queries and keys out of a fused projection
        dict(name="axes_train_B8_T4096_H6", op="axes_train", B=8, T=4096, H=6, Hk=6, D=128, R=128, dtype="bf16", kind="blocks", interleaved=False, fused=True),
        # fine-tuning in 32 bits, an odd length, the axes' pairs in turn, fewer keys than queries
        dict(name="axes_train_f32_B2_T1537_H8", op="axes_train", B=2, T=1537, H=8, Hk=2, D=128, R=128, dtype="f32", kind="turns", interleaved=False, fused=False),
        # one layer's gradients, as the repository's example trains it
        dict(name="clip_layer_W512", op="clip", layers=1, width=512, heads=4, dim=128, dtype="bf16", out="bf16", over=True),
        # a model's gradients, summed in 32 bits and clipped into the parameters' type
        dict(name="clip_model_L12_W2048", op="clip", layers=12, width=2048, heads=16, dim=128, dtype="f32", out="bf16", over=True),
        # a few sequences change places
        dict(name="swap_B3_H6", op="swap", B=3, H=6, K=128, V=128, more=2),
        # a serving batch is parked and another one resumed (268 MB of states each way)
        dict(name="swap_B256_H16", op="swap", B=256, H=16, K=128, V=128, more=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_train", "norm_train", "quant", "quant", "axes_fwd", "axes_train", "axes_train", "clip", "clip", "swap", "swap"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm_fwd", "norm_train", "quant"):
        step = rng.choice([8, 8, 128])
        D = step * _log(rng, 256 // step, 8192 // step)
        T = _log(rng, 1, min(32768, (1 << 25) // D))
        c = dict(op=op, B=_log(rng, 1, max(1, min(256, (1 << 25) // (D * T)))), T=T, D=D, dtype=dtype,
                 residual=rng.choice([dtype, dtype, "f32"]), fused=rng.random() < 0.3)
        if op == "quant":
            c["group"] = rng.choice([n for n in (0, 0, 32, 64, 128, 128) if n == 0 or D % n == 0])
        return c
    if op in ("axes_fwd", "axes_train"):
        H = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
        T = _log(rng, 1, 8192)
        D = rng.choice([32, 64, 96, 128, 128, 256])
        return dict(op=op, B=_log(rng, 1, max(1, min(256, 196608 // (H * T) * 128 // max(128, D)))), T=T, H=H,
                    Hk=rng.choice([n for n in range(1, H + 1) if H % n == 0]), D=D, R=rng.choice([D, D, D // 2]), dtype=dtype,
                    kind=rng.choice(["blocks", "uneven", "turns"]), interleaved=rng.random() < 0.3, fused=rng.random() < 0.5)
    if op == "clip":
        return dict(op=op, layers=_log(rng, 1, 24), width=_log(rng, 64, 1400), heads=rng.choice([1, 2, 4, 6, 8]), dim=rng.choice([32, 64, 96, 128]),
                    dtype=dtype, out=rng.choice([dtype, "bf16"]), over=rng.random() < 0.75)
    H = rng.choice([1, 2, 4, 6, 8, 16])
    B = _log(rng, 1, 4096 // H)
    return dict(op=op, B=B, H=H, K=rng.choice([16, 32, 64, 128, 128]), V=rng.choice([16, 32, 64, 128, 128]), more=rng.randint(0, 1 + B // 8))


def _sections(case):
    """How many of the R / 2 pairs turn by time, by height and by width."""
    n = case["R"] // 2
    if case["kind"] == "blocks":  # a quarter for the time, whole quarters of a 32-byte sector's pairs
        t = max(4, n // 16 * 4)
        h = (n - t) // 8 * 4
        return t, h, n - t - h
    if case["kind"] == "uneven":  # one pair more here and there
        t = n // 3 + 1
        h = (n - t) // 2
        return t, h, n - t - h
    h = n // 3 - n // 20
    return n - 2 * h, h, h


def _sizes(case):
    """The shapes of a model's gradients: the layers' parameters as the example layer has them, and a norm's weight."""
    w, inner = case["width"], case["heads"] * case["dim"]
    return [(4 * inner, w), (w, inner), (case["dim"],), (case["dim"],), (case["dim"],), (w,)] * case["layers"]


def prepare(case, seed):
    dev = torch.device("cuda")
    rng = torch.Generator(device=dev)
    rng.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=rng, device=dev) * std).to(dtype)

    s, op = dict(case=case), case["op"]
    if op in ("norm_fwd", "norm_train", "quant"):
        B, T, D, dt, rt = case["B"], case["T"], case["D"], DTYPES[case["dtype"]], DTYPES[case["residual"]]
        # a layer's output, and the sum of all before it, larger
        s["x"] = normal(B, T, 2 * D + 64, dtype=dt)[..., 64:64 + D] if case["fused"] else normal(B, T, D, dtype=dt)
        s["residual"] = normal(B, T, D, dtype=rt, std=3.0)
        s["w"] = normal(D, dtype=dt, std=0.1) + 1
        if op == "norm_train":
            s["dy"], s["dh"] = normal(B, T, D, dtype=dt), normal(B, T, D, dtype=rt)
    elif op in ("axes_fwd", "axes_train"):
        B, T, D, R, dt = case["B"], case["T"], case["D"], case["R"], DTYPES[case["dtype"]]

        def heads(n):
            if case["fused"]:
                return normal(B, T, 2 * n * D + 64, dtype=dt)[..., 64:64 + n * D].unflatten(-1, (n, D))
            return normal(B, T, n, D, dtype=dt)

        s["q"], s["k"] = heads(case["H"]), heads(case["Hk"])
        s["wq"], s["wk"] = normal(D, dtype=dt, std=0.1) + 1, normal(D, dtype=dt, std=0.1) + 1
        rows = max(T, 4096)
        angle = torch.arange(rows, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(R // 2, device=dev, dtype=torch.float64) * 2 / R)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["sections"] = _sections(case)
        # text, then frames of a side of 1 to 32, then text: the frames' time, row and column
        t = torch.arange(T, device=dev)
        side = min(32, max(1, math.isqrt(T // 4)))
        text = T // 8
        frames = torch.stack((text + (t - text) // (side * side), text + (t - text) % (side * side) // side, text + (t - text) % side))
        at = torch.where((t >= text) & (t < T - text), frames, t)
        start = torch.randint(0, rows - T + 1, (1, B, 1), generator=rng, device=dev)
        s["positions"] = (start + at[:, None]).to(torch.int32)
        if op == "axes_train":
            s["dq"], s["dk"] = normal(B, T, case["H"], D, dtype=dt), normal(B, T, case["Hk"], D, dtype=dt)
    elif op == "clip":
        dt = DTYPES[case["dtype"]]
        s["grads"] = [normal(*shape, dtype=dt, std=0.5 ** (i % 6)) for i, shape in enumerate(_sizes(case))]
        # one buffer that the optimiser reads, a parameter's part behind another's
        n = [g.numel() for g in s["grads"]]
        s["flat"] = torch.empty(sum(n), device=dev, dtype=DTYPES[case["out"]])
        s["out"] = [part.view(g.shape) for part, g in zip(s["flat"].split(n), s["grads"])]
        s["max_norm"] = 1.0 if case["over"] else 1e9
    else:
        B, H, K, V, n = case["B"], case["H"], case["K"], case["V"], 2 * case["B"] + case["more"] + 1
        s["states"] = normal(B, H, V, K) * torch.exp(normal(B, H, V, 1))
        s["cache"] = torch.randint(-127, 128, (n, H, V, K), generator=rng, device=dev, dtype=torch.int8)
        s["scales"] = torch.exp(normal(n, H, V)) / 127
        free = torch.randperm(n, generator=rng, device=dev)
        s["park"] = free[:B].to(torch.int32)
        # all that were parked just now, some that waited for longer, and a new sequence without a slot
        back = torch.cat((free[:B + case["more"]], torch.full((1,), -1, device=dev)))
        s["resume"] = back[torch.randperm(back.numel(), generator=rng, device=dev)].to(torch.int32)
    return s


# ---------------------------------------------------------------- plain forms

def _norm_grads(x, w, dn):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh, t = x * r, dn * w
    return r * (t - xh * (t * xh).mean(-1, keepdim=True)), (dn * xh).flatten(0, -2).sum(0)


def _plain_norm(s):
    case, dt, rt, w = s["case"], s["x"].dtype, s["residual"].dtype, s["w"].float()
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * w
    kept = h.to(rt)
    if case["op"] == "quant":
        g = y.unflatten(-1, (-1, case["group"] or case["D"]))
        scale = (g.abs().amax(-1, keepdim=True) / MOST).clamp(min=LEAST)
        return {"y": (g / scale).to(torch.float8_e4m3fn).flatten(-2), "scales": scale[..., 0], "h": kept}
    r = {"y": y.to(dt), "h": kept}
    if case["op"] == "norm_train":
        d, dw = _norm_grads(kept.float(), w, s["dy"].float())
        d = d + s["dh"].float()
        r.update(dx=d.to(dt), d_residual=d.to(rt), dw=dw.to(dt))
    return r


def _turn(x, c, s, interleaved):
    """The rotation of the first dimensions of each row by the angles of (c, s)."""
    n = c.shape[-1]
    if interleaved:
        x1, x2 = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack((x1 * c - x2 * s, x2 * c + x1 * s), -1).flatten(-2)
    else:
        x1, x2 = x[..., :n], x[..., n:2 * n]
        y = torch.cat((x1 * c - x2 * s, x2 * c + x1 * s), -1)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _plain_axes(s):
    case, dt, inter = s["case"], s["q"].dtype, s["case"]["interleaved"]
    i = torch.arange(case["R"] // 2, device=s["q"].device)
    a, b, c = s["sections"]
    if case["kind"] == "turns":
        axis = torch.where((i % 3 == 1) & (i // 3 < b), 1, torch.where((i % 3 == 2) & (i // 3 < c), 2, 0))
    else:
        axis = (i >= a).long() + (i >= a + b).long()
    at = s["positions"].long()[axis].permute(1, 2, 0)  # the position that each pair of a token turns by
    cos, sin = s["cos"][at, i][:, :, None], s["sin"][at, i][:, :, None]
    q, k, wq, wk = s["q"].float(), s["k"].float(), s["wq"].float(), s["wk"].float()

    def rows(x, w):
        return _turn(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w, cos, sin, inter).to(dt)

    r = {"q": rows(q, wq), "k": rows(k, wk)}
    if case["op"] == "axes_train":
        dq, dwq = _norm_grads(q, wq, _turn(s["dq"].float(), cos, -sin, inter))
        dk, dwk = _norm_grads(k, wk, _turn(s["dk"].float(), cos, -sin, inter))
        r.update(dq=dq.to(dt), dk=dk.to(dt), dwq=dwq.to(dt), dwk=dwk.to(dt))
    return r


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    by = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * by)
    return {"norm": norm, "out": s["flat"]}


def _plain_swap(s):
    x = s["states"]
    scale = (x.abs().amax(-1, keepdim=True) / 127).clamp(min=LEAST)
    park = s["park"].long()
    # the nearest whole number of steps: in 64 bits, as 32 lose it next to the middle between two
    s["cache"][park] = torch.round(x.double() / scale.double()).to(torch.int8)
    s["scales"][park] = scale[..., 0]
    at = s["resume"].long()
    known = (at >= 0) & (at < s["cache"].shape[0])
    at = torch.where(known, at, 0)
    back = s["cache"][at].float() * s["scales"][at][..., None]
    return {"states": back * known[:, None, None, None]}


# ------------------------------------------------------- the framework's calls

def _own_norm(s):
    from gated_delta_rule_19_gb300 import gdn
    case = s["case"]
    if case["op"] == "quant":
        return dict(zip(("y", "scales", "h"), gdn.gdn_add_norm_quant(s["x"], s["residual"], s["w"], eps=EPS, group=case["group"])))
    r = dict(zip(("y", "h"), gdn.gdn_add_norm_fwd(s["x"], s["residual"], s["w"], eps=EPS)))
    if case["op"] == "norm_train":
        r.update(zip(("dx", "d_residual", "dw"), gdn.gdn_add_norm_bwd(r["h"], s["w"], s["dy"], s["dh"], eps=EPS)))
    return r


def _own_axes(s):
    from gated_delta_rule_19_gb300 import gdn
    args = (s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"], s["sections"])
    how = dict(eps=EPS, interleaved=s["case"]["interleaved"], alternating=s["case"]["kind"] == "turns")
    r = dict(zip(("q", "k"), gdn.gdn_qk_norm_rope_axes_fwd(*args, **how)))
    if s["case"]["op"] == "axes_train":
        r.update(zip(("dq", "dk", "dwq", "dwk"), gdn.gdn_qk_norm_rope_axes_bwd(*args, s["dq"], s["dk"], **how)))
    return r


def _own_clip(s):
    from gated_delta_rule_19_gb300 import gdn
    return {"norm": gdn.gdn_clip_grads(s["grads"], s["max_norm"], out=s["out"]), "out": s["flat"]}


def _own_swap(s):
    from gated_delta_rule_19_gb300 import gdn
    gdn.gdn_state_store(s["states"], s["park"], s["cache"], s["scales"])
    return {"states": gdn.gdn_state_load(s["cache"], s["scales"], s["resume"])}


def run(state):
    kind = state["case"]["op"].split("_")[0]
    if own:
        return {"norm": _own_norm, "quant": _own_norm, "axes": _own_axes, "clip": _own_clip, "swap": _own_swap}[kind](state)
    return {"norm": _plain_norm, "quant": _plain_norm, "axes": _plain_axes, "clip": _plain_clip, "swap": _plain_swap}[kind](state)


# ---------------------------------------------------------- the work of a case

def _bytes(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_train", "quant"):
        rows, D, e, r = case["B"] * case["T"], case["D"], _bytes(case["dtype"]), _bytes(case["residual"])
        if op == "quant":  # x, residual in, the sum, 8 bits and the scales out
            return {"bytes": rows * (D * (e + 2 * r + 1) + 4 * (D // (case["group"] or D))) + D * e, "flops": rows * D * 8}
        b, f = rows * D * (2 * e + 2 * r) + D * e, rows * D * 5
        if op == "norm_train":  # the sum, dy, dh in, its gradient out (twice, where the types differ)
            b, f = b + rows * D * (e + 3 * r + (e if e != r else 0)) + 2 * D * e, f + rows * D * 12
        return {"bytes": b, "flops": f}
    if op in ("axes_fwd", "axes_train"):
        D, e, tokens = case["D"], _bytes(case["dtype"]), case["B"] * case["T"]
        rows, table = tokens * (case["H"] + case["Hk"]), tokens * (case["R"] * 4 + 12)  # a cosine and a sine for each pair, three positions
        b, f = rows * 2 * D * e + table + 2 * D * e, rows * (4 * D + 3 * case["R"])
        if op == "axes_train":
            b, f = b + rows * 3 * D * e + table + 4 * D * e, f + rows * (10 * D + 3 * case["R"])
        return {"bytes": b, "flops": f}
    if op == "clip":
        n = sum(math.prod(shape) for shape in _sizes(case))
        return {"bytes": n * (_bytes(case["dtype"]) + _bytes(case["out"])), "flops": 3 * n}
    n, back = (b * case["H"] * case["V"] for b in (case["B"], case["B"] + case["more"] + 1))
    return {"bytes": (n + back) * (5 * case["K"] + 4), "flops": 3 * n * case["K"] + back * case["K"]}


# ------------------------------------------------------------- in 64 bits

def _e4m3(x):
    """The nearest of e4m3's numbers (sign, four bits of exponent, three of mantissa), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-MOST, MOST)


def _axis_of(case, pair):
    a, b, c = _sections(case)
    if case["kind"] != "turns":
        return 0 if pair < a else 1 if pair < a + b else 2
    turn, place = pair % 3, pair // 3
    return turn if place < (a, b, c)[turn] else 0


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point()}
    if op in ("norm_fwd", "norm_train", "quant"):
        train = op == "norm_train"
        x, w = d["x"].requires_grad_(train), d["w"].requires_grad_(train)
        h = x + d["residual"]
        y = w * h / (h.pow(2).sum(-1, keepdim=True) / case["D"] + EPS).sqrt()
        if op == "quant":
            parts = y.split(case["group"] or case["D"], -1)
            scales = torch.stack([p.abs().max(-1).values for p in parts], -1) / MOST
            scales = torch.where(scales < LEAST, torch.full_like(scales, LEAST), scales)
            return {"y": torch.cat([_e4m3(p / scales[..., i, None]) for i, p in enumerate(parts)], -1), "scales": scales, "h": h}
        r = {"y": y, "h": h}
        if train:
            dx, dw = torch.autograd.grad((y, h), (x, w), (d["dy"], d["dh"]))
            r.update(dx=dx, d_residual=dx, dw=dw)
        return {n: t.detach() for n, t in r.items()}
    if op in ("axes_fwd", "axes_train"):
        train = op == "axes_train"
        n = case["R"] // 2
        by = torch.stack([torch.complex(d["cos"][:, i], d["sin"][:, i])[s["positions"][_axis_of(case, i)].long()] for i in range(n)], -1)[:, :, None]

        def rows(x, w):
            x = w * x / (x.pow(2).sum(-1, keepdim=True) / case["D"] + EPS).sqrt()
            z = x[..., :2 * n]
            z = z.unflatten(-1, (n, 2)) if case["interleaved"] else z.unflatten(-1, (2, n)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * by)
            return torch.cat((z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2), x[..., 2 * n:]), -1)

        ins = [d[i].requires_grad_(train) for i in ("q", "k", "wq", "wk")]
        q, k = rows(ins[0], ins[2]), rows(ins[1], ins[3])
        r = {"q": q, "k": k}
        if train:
            r.update(zip(("dq", "dk", "dwq", "dwk"), torch.autograd.grad((q, k), ins, (d["dq"], d["dk"]))))
        return {i: t.detach() for i, t in r.items()}
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.dot(g.double().flatten(), g.double().flatten())) for g in s["grads"]))
        by = min(1.0, s["max_norm"] / norm)
        return {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda"), "out": torch.cat([g.double().flatten() * by for g in s["grads"]])}
    parked = {int(n): b for b, n in enumerate(s["park"])}
    back = torch.zeros(s["resume"].numel(), *d["states"].shape[1:], dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["resume"].tolist()):
        if n in parked:
            x = d["states"][parked[n]]
            # the step is kept as a 32-bit number, and the steps are counted by what is kept
            step = (x.abs().max(-1, keepdim=True).values / 127).float().double()
            back[b] = torch.round(x / step) * step
        elif n >= 0:
            back[b] = s["cache"][n].double() * d["scales"][n][..., None]
    return {"states": back}
