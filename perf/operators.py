"""Measured cases of the sequence operators: the gated linear recurrence, the head norm with rotary
positions, and causal attention over packed episodes.

They are the mixing layers of a policy and critic over rollouts: what turns a rollout's steps into
the `values` and `log_rhos` that the credit-assignment estimators take. Each is measured as it is
used in training (forward and backward), over a whole prompt (forward) and for single steps.

`run` computes a case in elementary torch operations in 32 bits, or, where `own` is true, through
this package's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a recurrent layer's training step on 64 environments x 512 steps, episodes cut at about 1%
        dict(name="scan_train_64x512", op="scan_train", B=64, T=512, D=1024, dtype="bf16",
             p_reset=0.01, h0=True),
        # a small float32 layer with odd sizes
        dict(name="scan_train_odd_f32", op="scan_train", B=3, T=257, D=130, dtype="f32",
             p_reset=0.02, h0=False),
        # one very long sequence in a single forward pass
        dict(name="scan_prompt_131072", op="scan_prompt", B=1, T=131072, D=512, dtype="bf16",
             p_reset=0.0, h0=True),
        # acting: one step of 4096 environments' recurrent states
        dict(name="scan_step_4096", op="scan_step", B=4096, D=512, dtype="bf16", p_reset=0.01),
        # queries and keys of a training batch of 256 x 128 steps, whole heads rotated by halves
        dict(name="norm_train_32768", op="norm_train", tokens=32768, Hq=16, Hk=4, D=128, R=128,
             interleaved=False, dtype="bf16", max_pos=1024),
        # float32 heads of an odd width, rotated in part, in interleaved pairs
        dict(name="norm_train_odd_f32", op="norm_train", tokens=4999, Hq=6, Hk=3, D=80, R=20,
             interleaved=True, dtype="f32", max_pos=5000),
        # acting: one new token for each of 64 environments, at positions of a long context
        dict(name="norm_prompt_64", op="norm_prompt", tokens=64, Hq=16, Hk=4, D=128, R=128,
             interleaved=False, dtype="bf16", max_pos=131072),
        # training on packed episodes of 0 to 1024 steps, 64-wide heads shared by three
        dict(name="attn_train_packed", op="attn_train", nseq=48, max_len=1024, ragged=True, Hq=12,
             Hk=4, D=64, lens_seed=7),
        # training on two long episodes
        dict(name="attn_train_4096", op="attn_train", nseq=2, max_len=4096, ragged=False, Hq=16,
             Hk=4, D=128, lens_seed=0),
        # one whole long prompt, all query heads on one key/value head
        dict(name="attn_prompt_16384", op="attn_prompt", nseq=1, max_len=16384, ragged=False, Hq=8,
             Hk=1, D=128, lens_seed=0),
        # acting: one new token for each of 64 environments over caches of up to 8192 steps
        dict(name="attn_step_64x8192", op="attn_step", B=64, S=8192, Hq=16, Hk=4, D=128,
             lens_seed=3),
        # acting: one environment, a short cache
        dict(name="attn_step_1x1024", op="attn_step", B=1, S=1024, Hq=4, Hk=2, D=64, lens_seed=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_train", "scan_prompt", "scan_step", "norm_train", "norm_prompt",
                     "attn_train", "attn_prompt", "attn_step"])
    if op in ("scan_train", "scan_prompt"):
        D = _log(rng, 64, 2048)
        T = _log(rng, 1, 131072 if op == "scan_prompt" else 4096)
        B = max(1, min(_log(rng, 1, 128), (1 << 25) // (T * D)))
        return dict(op=op, B=B, T=T, D=D, dtype=rng.choice(["bf16", "f32"]),
                    p_reset=rng.choice([0.0, 0.001, 0.02]), h0=rng.random() < 0.5)
    if op == "scan_step":
        return dict(op=op, B=_log(rng, 1, 4096), D=_log(rng, 64, 2048),
                    dtype=rng.choice(["bf16", "f32"]), p_reset=rng.choice([0.0, 0.01]))
    if op in ("norm_train", "norm_prompt"):
        Hk = rng.choice([1, 2, 3, 4, 8])
        D = rng.choice([32, 64, 80, 96, 128])
        tokens = _log(rng, 1, 32768 if op == "norm_train" else 65536)
        tokens = max(1, min(tokens, (1 << 26) // (4 * Hk * D)))
        return dict(op=op, tokens=tokens, Hq=Hk * rng.choice([1, 2, 3, 4]), Hk=Hk, D=D,
                    R=rng.choice([D, D // 2, D // 4]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f32"]), max_pos=_log(rng, 512, 131072))
    Hk = rng.choice([1, 2, 3, 4])
    group = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 128])
    if op == "attn_step":
        S = _log(rng, 16, 16384)
        B = max(1, min(_log(rng, 1, 128), (1 << 21) // (S * Hk)))
        return dict(op=op, B=B, S=S, Hq=Hk * group, Hk=Hk, D=D, lens_seed=rng.randrange(1 << 20))
    max_len = _log(rng, 1, 4096 if op == "attn_train" else 8192)
    room = (1 << (29 if op == "attn_train" else 31)) // (max_len * (max_len + 1024) * Hk * group)
    return dict(op=op, nseq=max(1, min(_log(rng, 1, 64), room)), max_len=max_len,
                ragged=rng.random() < 0.7, Hq=Hk * group, Hk=Hk, D=D,
                lens_seed=rng.randrange(1 << 20))


def _lengths(case):
    """Lengths of the packed episodes (zero among them), or of the caches."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "attn_step":
        return [r.randint(max(1, case["S"] // 16), case["S"]) for _ in range(case["B"])]
    if not case["ragged"]:
        return [case["max_len"]] * case["nseq"]
    lens = [r.randint(0, case["max_len"]) for _ in range(case["nseq"])]
    lens[r.randrange(len(lens))] = case["max_len"]
    return lens


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    dt = DTYPES[case.get("dtype", "bf16")]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(shape, device="cuda", generator=g) * scale + shift).to(dtype)

    def flags(*shape, p):
        return torch.rand(shape, device="cuda", generator=g) < p

    s = {"op": op, "case": dict(case)}
    if op.startswith("scan"):
        B, D = case["B"], case["D"]
        shape = (B, D) if op == "scan_step" else (B, case["T"], D)
        s["x"] = normal(*shape)
        s["gate"] = normal(*shape, scale=1.5, shift=2.0)
        s["reset"] = flags(*shape[:-1], p=case["p_reset"]) if case["p_reset"] else None
        if op == "scan_step":
            s["state"] = normal(B, D, dtype=torch.float32)
            return s
        s["h0"] = normal(B, D, dtype=torch.float32) if case["h0"] else None
        if op == "scan_train":
            s["dh"] = normal(*shape)
        return s
    if op.startswith("norm"):
        n, Hq, Hk, D, R = (case[k] for k in ("tokens", "Hq", "Hk", "D", "R"))
        qkv = normal(n, (Hq + 2 * Hk) * D)  # the fused projection's output
        s["q"] = qkv[:, :Hq * D].view(n, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(n, Hk, D)
        s["q_weight"] = normal(D, scale=0.1, shift=1.0, dtype=torch.float32)
        s["k_weight"] = normal(D, scale=0.1, shift=1.0, dtype=torch.float32)
        s["positions"] = torch.randint(0, case["max_pos"], (n,), device="cuda", generator=g,
                                       dtype=torch.int32)
        inv = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        ang = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        if op == "norm_train":
            s["dq"], s["dk"] = normal(n, Hq, D), normal(n, Hk, D)
        return s
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    lens = _lengths(case)
    if op == "attn_step":
        B, S = case["B"], case["S"]
        s["q"] = normal(B, Hq, D)
        s["k_cache"], s["v_cache"] = normal(B, S, Hk, D), normal(B, S, Hk, D)
        s["lengths"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        return s
    total = sum(lens)
    s["q"], s["k"] = normal(total, Hq, D), normal(total, Hk, D)
    qkv = normal(total, (Hq + 2 * Hk) * D)  # values are a view of the fused projection's output
    s["v"] = qkv[:, (Hq + Hk) * D:].view(total, Hk, D)
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    s["cu_seqlens"] = torch.tensor(ends, device="cuda", dtype=torch.int32)
    # the padded layout that the elementary form works in: token of (sequence, place), and back
    L = case["max_len"]
    lt = torch.tensor(lens, device="cuda")
    place = torch.arange(L, device="cuda")
    s["valid"] = place[None, :] < lt[:, None]
    s["token"] = (s["cu_seqlens"][:-1, None] + place[None, :]).long().masked_fill(~s["valid"], 0)
    if op == "attn_train":
        s["dout"] = normal(total, Hq, D)
    return s


# ---------------------------------------------------------------------------
# Elementary forms, in 32 bits
# ---------------------------------------------------------------------------
def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, by doubling spans."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat([b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _scan_forward(s):
    x, a = s["x"].float(), 1.0 / (1.0 + torch.exp(-s["gate"].float()))
    carry = a if s["reset"] is None else a * (~s["reset"]).float()[..., None]
    b = (1.0 - a) * x
    if s["h0"] is not None:
        b = torch.cat([b[:, :1] + carry[:, :1] * s["h0"][:, None], b[:, 1:]], 1)
    return x, a, carry, _doubling(carry, b)


def _scan_train(s):
    dt = s["x"].dtype
    x, a, carry, h = _scan_forward(s)
    up = torch.cat([carry[:, 1:], torch.zeros_like(carry[:, :1])], 1)
    lam = _doubling(up.flip(1), s["dh"].float().flip(1)).flip(1)
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    prev = torch.cat([first, h[:, :-1]], 1)
    if s["reset"] is not None:
        prev = prev * (~s["reset"]).float()[..., None]
    dx = (1.0 - a) * lam
    dg = a * (1.0 - a) * lam * (prev - x)
    return h.to(dt), h[:, -1], dx.to(dt), dg.to(dt), carry[:, 0] * lam[:, 0]


def _scan_step(s):
    x, a = s["x"].float(), 1.0 / (1.0 + torch.exp(-s["gate"].float()))
    carry = a if s["reset"] is None else a * (~s["reset"]).float()[..., None]
    h = carry * s["state"] + (1.0 - a) * x
    return h.to(s["x"].dtype), h


def _rotate(u, c, sn, interleaved):
    R = 2 * c.shape[-1]
    head, tail = u[..., :R], u[..., R:]
    if interleaved:
        u1, u2 = head[..., 0::2], head[..., 1::2]
        y = torch.stack([u1 * c - u2 * sn, u2 * c + u1 * sn], -1).flatten(-2)
    else:
        u1, u2 = head[..., :R // 2], head[..., R // 2:]
        y = torch.cat([u1 * c - u2 * sn, u2 * c + u1 * sn], -1)
    return torch.cat([y, tail], -1)


def _norm_rope(x, w, c, sn, interleaved):
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    return _rotate(xf * r * w, c, sn, interleaved).to(x.dtype)


def _norm_rope_backward(dy, x, w, c, sn, interleaved):
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    du = _rotate(dy.float(), c, -sn, interleaved)
    dw = (du * xf * r).sum((0, 1))
    t = du * w
    dx = r * (t - xf * r * r * (t * xf).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _norm(s, train):
    inter = s["case"]["interleaved"]
    p = s["positions"].long()
    c, sn = s["cos"][p][:, None], s["sin"][p][:, None]
    out = [_norm_rope(s["q"], s["q_weight"], c, sn, inter),
           _norm_rope(s["k"], s["k_weight"], c, sn, inter)]
    if train:
        dq, dqw = _norm_rope_backward(s["dq"], s["q"], s["q_weight"], c, sn, inter)
        dk, dkw = _norm_rope_backward(s["dk"], s["k"], s["k_weight"], c, sn, inter)
        out += [dq, dk, dqw, dkw]
    return tuple(out)


def _attention(s, train):
    q, k, v = s["q"], s["k"], s["v"]
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    scale = D ** -0.5
    tok, valid = s["token"], s["valid"]
    n, L = tok.shape

    def padded(t):  # [n, H, L, D]
        x = t.float()[tok] * valid[..., None, None]
        return x.transpose(1, 2)

    def packed(x, dtype):  # back to [tokens, H, D]
        return x.transpose(1, 2)[valid].to(dtype)

    qp, kp, vp = padded(q), padded(k), padded(v)
    kp, vp = (t.repeat_interleave(Hq // Hk, 1) for t in (kp, vp))
    place = torch.arange(L, device=q.device)
    seen = (place[None, :] <= place[:, None])[None, None] & valid[:, None, None, :]
    sc = (qp @ kp.transpose(2, 3)) * scale
    sc = sc.masked_fill(~seen, float("-inf"))
    m = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(sc - m)
    del sc
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = p @ vp
    out = packed(o, q.dtype)
    if not train:
        return out
    do = padded(s["dout"])
    dv = p.transpose(2, 3) @ do
    ds = do @ vp.transpose(2, 3)
    ds = p * (ds - (do * o).sum(-1, keepdim=True))
    del p
    dq = (ds @ kp) * scale
    dk = (ds.transpose(2, 3) @ qp) * scale
    shared = (n, Hk, Hq // Hk, L, D)
    return (out, packed(dq, q.dtype), packed(dk.view(shared).sum(2), k.dtype),
            packed(dv.view(shared).sum(2), v.dtype))


def _attention_step(s):
    q, kc, vc = s["q"], s["k_cache"], s["v_cache"]
    B, S, Hk, D = kc.shape
    Hq = q.shape[1]
    qf = q.float().view(B, Hk, Hq // Hk, D)
    kf, vf = kc.float().transpose(1, 2), vc.float().transpose(1, 2)
    sc = (qf @ kf.transpose(2, 3)) * D ** -0.5
    seen = torch.arange(S, device=q.device)[None, :] < s["lengths"][:, None]
    sc = sc.masked_fill(~seen[:, None, None], float("-inf"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    return (p @ vf).reshape(B, Hq, D).to(q.dtype)


def _plain(s):
    op = s["op"]
    if op == "scan_train":
        return _scan_train(s)
    if op == "scan_prompt":
        h = _scan_forward(s)[3]
        return h.to(s["x"].dtype), h[:, -1]
    if op == "scan_step":
        return _scan_step(s)
    if op.startswith("norm"):
        return _norm(s, op == "norm_train")
    if op == "attn_step":
        return _attention_step(s)
    return _attention(s, op == "attn_train")


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _framework(s):
    import linear_recurrence_scan_affine_gb300 as rl
    op = s["op"]
    if op in ("scan_train", "scan_prompt"):
        h, last = rl.rlcs_gated_scan(s["x"], s["gate"], reset=s["reset"], h0=s["h0"])
        if op == "scan_prompt":
            return h, last
        dx, dg, dh0 = rl.rlcs_gated_scan_backward(s["dh"], s["x"], s["gate"], h, reset=s["reset"],
                                                  h0=s["h0"])
        return h, last, dx, dg, dh0
    if op == "scan_step":
        return rl.rlcs_gated_step(s["x"], s["gate"], s["state"], reset=s["reset"])
    if op.startswith("norm"):
        args = (s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos"], s["sin"], s["positions"])
        kw = dict(eps=EPS, interleaved=s["case"]["interleaved"])
        out = rl.rlcs_qk_norm_rope(*args, **kw)
        if op == "norm_train":
            out += rl.rlcs_qk_norm_rope_backward(s["dq"], s["dk"], *args, **kw)
        return out
    if op == "attn_step":
        return rl.rlcs_attention_step(s["q"], s["k_cache"], s["v_cache"], s["lengths"])
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu_seqlens"]
    if op == "attn_prompt":
        return rl.rlcs_attention(q, k, v, cu)
    out, lse = rl.rlcs_attention(q, k, v, cu, return_lse=True)
    return (out,) + rl.rlcs_attention_backward(s["dout"], q, k, v, out, lse, cu)


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# Work of one pass
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    e = 4 if case.get("dtype") == "f32" else 2
    if op.startswith("scan"):
        B, T, D = case["B"], case.get("T", 1), case["D"]
        n = B * T * D
        reset = B * T if case["p_reset"] else 0
        if op == "scan_step":
            return {"bytes": n * (3 * e + 8) + reset, "flops": 12 * n}
        ends = 4 * B * D * (2 if case["h0"] else 1)
        if op == "scan_prompt":
            return {"bytes": 3 * e * n + reset + ends, "flops": 12 * n}
        # the gradient's inputs are the outputs' gradients and the forward's inputs, read once
        return {"bytes": 9 * e * n + 2 * reset + 2 * ends, "flops": 30 * n}
    if op.startswith("norm"):
        n, heads, D, R = case["tokens"], case["Hq"] + case["Hk"], case["D"], case["R"]
        table = 4 * R * min(n, case["max_pos"]) + 4 * n
        elems = n * heads * D
        if op == "norm_prompt":
            return {"bytes": 2 * e * elems + table, "flops": 8 * elems}
        return {"bytes": 5 * e * elems + 2 * table, "flops": 28 * elems}
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    lens = _lengths(case)
    if op == "attn_step":
        n = sum(lens)
        return {"bytes": 4 * n * Hk * D + 4 * case["B"] * Hq * D, "flops": 4 * n * Hq * D}
    n, pairs = sum(lens), sum(x * (x + 1) // 2 for x in lens)
    forward = {"bytes": 2 * n * D * (2 * Hq + 2 * Hk), "flops": 4 * pairs * Hq * D}
    if op == "attn_prompt":
        return forward
    return {"bytes": forward["bytes"] + 2 * n * D * (4 * Hq + 4 * Hk),
            "flops": 14 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, step by step
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    f = {k: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t)
         for k, t in s.items()}
    op = case["op"]
    if op.startswith("scan"):
        return _exact_scan(op, f)
    if op.startswith("norm"):
        return _exact_norm(op, f, case)
    if op == "attn_step":
        out = torch.empty_like(f["q"])
        group = case["Hq"] // case["Hk"]
        for b, n in enumerate(_lengths(case)):
            for h in range(case["Hk"]):
                rows = slice(h * group, (h + 1) * group)
                w = torch.softmax(f["q"][b, rows] @ f["k_cache"][b, :n, h].T
                                  / math.sqrt(case["D"]), 1)
                out[b, rows] = w @ f["v_cache"][b, :n, h]
        return out
    return _exact_attention(op, f, case)


def _exact_scan(op, f):
    x, gate, reset = f["x"], f["gate"], f["reset"]
    a = torch.sigmoid(gate)
    if op == "scan_step":
        old = f["state"] if reset is None else torch.where(reset[:, None], 0.0, f["state"])
        h = a * old + torch.sigmoid(-gate) * x
        return h, h
    T = x.shape[1]
    h = torch.empty_like(x)
    before = torch.empty_like(x)
    cur = torch.zeros_like(x[:, 0]) if f["h0"] is None else f["h0"]
    keep = torch.ones_like(x[:, :, :1]) if reset is None else 1.0 - reset.double()[:, :, None]
    b = torch.sigmoid(-gate) * x
    for t in range(T):
        before[:, t] = cur * keep[:, t]
        cur = torch.addcmul(b[:, t], a[:, t], before[:, t])
        h[:, t] = cur
    if op == "scan_prompt":
        return h, cur
    lam = torch.empty_like(x)
    cur = torch.zeros_like(x[:, 0])
    for t in range(T - 1, -1, -1):
        lam[:, t] = f["dh"][:, t] + cur
        cur = a[:, t] * keep[:, t] * lam[:, t]
    slope = a * torch.sigmoid(-gate)
    return h, h[:, -1], torch.sigmoid(-gate) * lam, slope * lam * (before - x), cur


def _exact_norm(op, f, case):
    R, inter = case["R"], case["interleaved"]
    D = case["D"]
    # the rotation of each token as one D x D matrix acting on its heads
    i = torch.arange(R // 2, device="cuda")
    one, two = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
    out, grads, wgrads = [], [], []
    for name in ("q", "k"):
        x, w = f[name], f[name + "_weight"]
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dx, dw = torch.empty_like(y), torch.zeros(D, dtype=torch.float64, device="cuda")
        for lo in range(0, x.shape[0], 1024):
            at = slice(lo, lo + 1024)
            p = f["positions"][at].long()
            M = torch.eye(D, dtype=torch.float64, device="cuda").repeat(len(p), 1, 1)
            M[:, one, one], M[:, one, two] = f["cos"][p], -f["sin"][p]
            M[:, two, one], M[:, two, two] = f["sin"][p], f["cos"][p]
            xs = x[at]
            ms = xs.square().mean(-1, keepdim=True) + EPS
            y[at] = (xs / ms.sqrt() * w) @ M.transpose(1, 2)
            if op == "norm_train":
                du = f["d" + name][at] @ M
                unit = xs / ms.sqrt()
                dw += (du * unit).sum((0, 1))
                dunit = du * w
                dx[at] = (dunit - unit * (dunit * unit).mean(-1, keepdim=True)) / ms.sqrt()
        out.append(y)
        grads.append(dx)
        wgrads.append(dw)
    return tuple(out + grads + wgrads) if op == "norm_train" else tuple(out)


def _exact_attention(op, f, case):
    q, k, v = f["q"], f["k"], f["v"]
    group = case["Hq"] // case["Hk"]
    out = torch.empty_like(q)
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros(
        k.shape, dtype=torch.float64, device="cuda")
    at = 0
    for n in _lengths(case):
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for h in range(case["Hq"]):
            kv = h // group
            w = (q[rows, h] @ k[rows, kv].T / math.sqrt(case["D"])).masked_fill(later, -math.inf)
            w = torch.softmax(w, 1)
            out[rows, h] = w @ v[rows, kv]
            if op == "attn_train":
                g = f["dout"][rows, h]
                dv[rows, kv] += w.T @ g
                t = g @ v[rows, kv].T
                t = w * (t - (t * w).sum(1, keepdim=True)) / math.sqrt(case["D"])
                dq[rows, h] = t @ k[rows, kv]
                dk[rows, kv] += t.T @ q[rows, h]
    return out if op == "attn_prompt" else (out, dq, dk, dv)
