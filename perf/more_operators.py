"""Measured cases of linear attention with a decay per head, the clipped policy loss and distillation
from a teacher's top logits.

Linear attention is the mixing layer whose whole past is one matrix per head; the two losses are what
a policy over a set of actions (or a vocabulary) learns from: the advantages that the estimators give,
and the largest logits of a teacher. Each is measured as it is used in training (forward and
backward), forward alone (whole prompts, evaluation) and, where it acts, for single steps.

`run` computes a case in elementary torch operations in 32 bits, or, where `own` is true, through
this package's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CLIP = 0.2


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # linear attention: a layer's training step on eight rollouts of 4096 steps
        dict(name="linear_train_8x4096", op="linear_train", nseq=8, max_len=4096, ragged=False,
             Hq=16, Hk=16, D=128, state=False, lens_seed=0),
        # training on packed episodes of 0 to 1024 steps, 64-wide heads, states shared by three
        dict(name="linear_train_packed", op="linear_train", nseq=48, max_len=1024, ragged=True,
             Hq=12, Hk=4, D=64, state=True, lens_seed=7),
        # one very long sequence read in, its last state kept for acting
        dict(name="linear_prompt_131072", op="linear_prompt", nseq=1, max_len=131072, ragged=False,
             Hq=8, Hk=8, D=128, state=False, lens_seed=0),
        # 64 short pieces of up to 200 steps, read in on top of the states they continue
        dict(name="linear_prompt_64x200", op="linear_prompt", nseq=64, max_len=200, ragged=True,
             Hq=16, Hk=4, D=128, state=True, lens_seed=3),
        # acting: one step of 256 environments
        dict(name="linear_step_256", op="linear_step", B=256, Hq=16, Hk=16, D=128, p_reset=0.01),
        # acting: one environment
        dict(name="linear_step_1", op="linear_step", B=1, Hq=4, Hk=2, D=64, p_reset=0.0),
        # policy update over a vocabulary, a quarter of the tokens not the policy's own
        dict(name="policy_train_16384x32768", op="policy_train", tokens=16384, V=32768,
             dtype="bf16", p_mask=0.25, illegal=0.0, kl=0.05, entropy=0.0),
        # policy update of 4096 environments x 128 steps with few actions, some of them illegal
        dict(name="policy_train_4096x128x6", op="policy_train", tokens=524288, V=6, dtype="f32",
             p_mask=0.0, illegal=0.2, kl=0.0, entropy=0.01),
        # log probabilities and losses without a gradient, rows of an odd length
        dict(name="policy_eval_997x50001", op="policy_eval", tokens=997, V=50001, dtype="bf16",
             p_mask=0.1, illegal=0.0, kl=0.05, entropy=0.01),
        # distillation over a large vocabulary from a teacher's 64 largest logits
        dict(name="distill_train_4096x131072", op="distill_train", tokens=4096, V=131072, K=64,
             dtype="bf16", p_mask=0.0, p_absent=0.0, whole=True, temperature=1.0),
        # a small float32 student, odd sizes, softened, some entries absent
        dict(name="distill_train_odd_f32", op="distill_train", tokens=1023, V=31999, K=17,
             dtype="f32", p_mask=0.2, p_absent=0.1, whole=False, temperature=2.0),
        # evaluating a student on a few tokens
        dict(name="distill_eval_64", op="distill_eval", tokens=64, V=8192, K=8, dtype="bf16",
             p_mask=0.0, p_absent=0.0, whole=False, temperature=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear_train", "linear_prompt", "linear_step", "policy_train", "policy_eval",
                     "distill_train", "distill_eval"])
    if op.startswith("linear"):
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hk * rng.choice([1, 1, 2, 3, 4])
        D = rng.choice([32, 64, 64, 96, 128, 128])
        if op == "linear_step":
            B = max(1, min(_log(rng, 1, 1024), (1 << 26) // (Hk * D * D)))
            return dict(op=op, B=B, Hq=Hq, Hk=Hk, D=D, p_reset=rng.choice([0.0, 0.02]))
        max_len = _log(rng, 1, 4096 if op == "linear_train" else 65536)
        room = (1 << (25 if op == "linear_train" else 26)) // (max_len * Hq * D)
        return dict(op=op, nseq=max(1, min(_log(rng, 1, 128), room)), max_len=max_len,
                    ragged=rng.random() < 0.7, Hq=Hq, Hk=Hk, D=D, state=rng.random() < 0.5,
                    lens_seed=rng.randrange(1 << 20))
    V = _log(rng, 2, 131072)
    tokens = max(1, min(_log(rng, 1, 1 << 19), (1 << 28) // V))
    common = dict(op=op, tokens=tokens, V=V, dtype=rng.choice(["bf16", "f32"]),
                  p_mask=rng.choice([0.0, 0.1, 0.5]))
    if op.startswith("policy"):
        return dict(common, illegal=rng.choice([0.0, 0.0, 0.3]), kl=rng.choice([0.0, 0.05]),
                    entropy=rng.choice([0.0, 0.01]))
    return dict(common, K=min(V, _log(rng, 1, 256)), p_absent=rng.choice([0.0, 0.2]),
                whole=rng.random() < 0.5, temperature=rng.choice([1.0, 1.0, 2.0, 0.7]))


def _lengths(case):
    """Lengths of the packed episodes, zero among them."""
    if not case["ragged"]:
        return [case["max_len"]] * case["nseq"]
    r = random.Random(case["lens_seed"])
    lens = [r.randint(0, case["max_len"]) for _ in range(case["nseq"])]
    lens[r.randrange(len(lens))] = case["max_len"]
    return lens


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
CHUNK = 64  # tokens to a chunk of the elementary form
ROWS = 1 << 27  # elements of logits made at a time


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"op": case["op"], "case": dict(case)}
    if case["op"].startswith("linear"):
        _prepare_linear(s, case, g)
    else:
        _prepare_logits(s, case, g)
    return s


def _normal(g, *shape, scale=1.0, shift=0.0, dtype=torch.bfloat16):
    return (torch.randn(shape, device="cuda", generator=g) * scale + shift).to(dtype)


def _prepare_linear(s, case, g):
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    # decays from 0.7 to 0.999 a step, spread over the heads as such layers have them
    spread = torch.rand(Hk, device="cuda", generator=g, dtype=torch.float64)
    s["log_decay"] = -(0.36 * (1.0 / 360.0) ** spread).float()
    if case["op"] == "linear_step":
        B = case["B"]
        s["q"], s["k"], s["v"] = _normal(g, B, Hq, D), _normal(g, B, Hk, D), _normal(g, B, Hk, D)
        s["state"] = _normal(g, B, Hk, D, D, scale=2.0, dtype=torch.float32)
        s["reset"] = (torch.rand(B, device="cuda", generator=g) < case["p_reset"]
                      if case["p_reset"] else None)
        return
    lens = _lengths(case)
    n, total = len(lens), sum(lens)
    s["q"], s["k"] = _normal(g, total, Hq, D), _normal(g, total, Hk, D)
    qkv = _normal(g, total, (Hq + 2 * Hk) * D)  # values are a view of the fused projection's output
    s["v"] = qkv[:, (Hq + Hk) * D:].view(total, Hk, D)
    ends = [0]
    for m in lens:
        ends.append(ends[-1] + m)
    s["cu_seqlens"] = torch.tensor(ends, device="cuda", dtype=torch.int32)
    s["state"] = (_normal(g, n, Hk, D, D, scale=2.0, dtype=torch.float32) if case["state"]
                  else None)
    if case["op"] == "linear_train":
        s["dout"] = _normal(g, total, Hq, D)
        s["dlast"] = _normal(g, n, Hk, D, D, dtype=torch.float32) if case["state"] else None
    # the padded layout that the elementary form works in: token of (sequence, place), and back
    L = -(-max(lens) // CHUNK) * CHUNK
    lt = torch.tensor(lens, device="cuda")
    place = torch.arange(L, device="cuda")
    s["lens"], s["valid"] = lt, place[None, :] < lt[:, None]
    s["token"] = (s["cu_seqlens"][:-1, None] + place[None, :]).long().masked_fill(~s["valid"], 0)


def _prepare_logits(s, case, g):
    n, V, dt = case["tokens"], case["V"], DTYPES[case["dtype"]]
    s["logits"] = torch.empty(n, V, device="cuda", dtype=dt)
    s["mask"] = (torch.rand(n, device="cuda", generator=g) >= case["p_mask"] if case["p_mask"]
                 else None)
    s["dloss"] = torch.full((n,), 1.0 / n, device="cuda")
    policy = case["op"].startswith("policy")
    if policy:
        s["actions"] = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
        s["advantages"] = _normal(g, n, dtype=torch.float32)
        s["old_logp"] = torch.empty(n, device="cuda")
        s["ref_logp"] = torch.empty(n, device="cuda") if case["kl"] else None
    else:
        K = case["K"]
        gaps = torch.randint(1, V // K + 1, (n, K), device="cuda", generator=g).cumsum(1)
        start = torch.randint(0, V, (n, 1), device="cuda", generator=g)
        ids = (start + gaps) % V  # distinct, as a teacher's are
        drops = torch.rand(n, K, device="cuda", generator=g)
        s["top_logits"] = 6.0 - (drops * min(0.5, 8.0 / K)).cumsum(1)
        lse = torch.logsumexp(s["top_logits"].double() / case["temperature"], 1)
        more = 0.3 * torch.rand(n, device="cuda", generator=g)  # what the rest of the row weighs
        s["teacher_lse"] = (lse + more).float() if case["whole"] else None
        s["top_ids"] = ids.to(torch.int32)
        if case["p_absent"]:
            absent = torch.rand(n, K, device="cuda", generator=g) < case["p_absent"]
            s["top_ids"] = s["top_ids"].masked_fill(absent, -1)
    step = max(1, ROWS // V)
    for lo in range(0, n, step):
        x = torch.randn(min(step, n - lo), V, device="cuda", generator=g) * 2.0
        at = slice(lo, lo + x.shape[0])
        if not policy:
            x.scatter_add_(1, ids[at], s["top_logits"][at] * 0.5)
            s["logits"][at] = x.to(dt)
            continue
        a = s["actions"][at].long()[:, None]
        if case["illegal"]:
            bad = torch.rand(x.shape, device="cuda", generator=g) < case["illegal"]
            x.masked_fill_(bad.scatter_(1, a, False), -math.inf)
        x.scatter_add_(1, a, 3.0 * torch.rand(a.shape, device="cuda", generator=g))
        x = x.to(dt)
        s["logits"][at] = x
        x = x.float()
        logp = (x.gather(1, a)[:, 0].double() - torch.logsumexp(x, 1).double())
        # log ratios of a few updates; none within 1e-3 of where clipping sets in, since there the
        # gradient jumps and a rounding of the log probability decides
        off = _normal(g, len(logp), scale=0.15, dtype=torch.float64)
        for edge in (math.log(1.0 - CLIP), math.log(1.0 + CLIP)):
            off = torch.where((off - edge).abs() < 1e-3, torch.full_like(off, edge + 2e-3), off)
        s["old_logp"][at] = (logp - off).float()
        if case["kl"]:
            s["ref_logp"][at] = (logp + _normal(g, len(logp), scale=0.3,
                                                dtype=torch.float64)).float()


# ---------------------------------------------------------------------------
# Elementary forms, in 32 bits
# ---------------------------------------------------------------------------
def _powers(log_decay, steps):
    """decay ** steps, its exponents in 64 bits: log_decay [Hk], steps [n, ...] -> [n, Hk, ...]."""
    ld = log_decay.double().view(1, -1, *([1] * (steps.dim() - 1)))
    return torch.exp(ld * steps[:, None].double()).float()


def _linear(s, train):
    q, k, v = s["q"], s["k"], s["v"]
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    G, scale, ld = Hq // Hk, D ** -0.5, s["log_decay"]
    tok, valid = s["token"], s["valid"]
    n, L = tok.shape
    C, nc = CHUNK, L // CHUNK

    def padded(t):  # [n, Hk, nc, heads sharing a state, C, D]
        x = t.float()[tok] * valid[..., None, None]
        return x.view(n, nc, C, Hk, -1, D).permute(0, 3, 1, 4, 2, 5)

    def packed(x, dtype):  # back to [tokens, heads, D]
        x = x.permute(0, 2, 4, 1, 3, 5).reshape(n, L, -1, D)
        return x[valid].to(dtype)

    i = torch.arange(C, device=q.device)
    begin = (torch.arange(nc, device=q.device)[None] * C).minimum(s["lens"][:, None])  # [n, nc]
    held = s["lens"][:, None] - begin
    held = held.clamp(max=C)  # tokens of each chunk
    end = begin + held
    later = (i[:, None] - i[None, :]).clamp(min=0)[None]
    M = _powers(ld, later)[:, :, None, None] * (i[:, None] >= i[None, :])  # [1, Hk, 1, 1, C, C]
    into = _powers(ld, (i + 1)[None])[:, :, None, None, :, None]  # from a chunk's start to its rows
    left = (held[..., None] - 1 - i).clamp(min=0)  # from its rows to its end
    out_of = _powers(ld, left)[:, :, :, None, :, None]
    # how much of one chunk's end is left at a later one's start
    apart = (begin[:, :, None] - end[:, None, :]).clamp(min=0)
    earlier = torch.ones(nc, nc, device=q.device).tril(-1)
    carry = _powers(ld, apart) * earlier  # [n, Hk, nc, nc]
    start, whole = _powers(ld, begin), _powers(ld, s["lens"][:, None])[..., 0]

    qp, kp, vp = padded(q) * scale, padded(k), padded(v)
    own_state = ((kp * out_of).transpose(-1, -2) @ vp)[:, :, :, 0]  # [n, Hk, nc, D, D]
    before = (carry @ own_state.flatten(-2)).view_as(own_state)
    if s["state"] is not None:
        before = before + start[..., None, None] * s["state"][:, :, None]
    score = (qp @ kp.transpose(-1, -2)) * M
    o = packed(score @ vp + (qp * into) @ before[:, :, :, None], q.dtype)
    if not train:
        rest = _powers(ld, s["lens"][:, None] - end)  # from each chunk's end to the last token
        last = (own_state * rest[..., None, None]).sum(2)
        if s["state"] is not None:
            last = last + whole[..., None, None] * s["state"]
        return o, last
    do = padded(s["dout"])
    dscore = (do @ vp.transpose(-1, -2)) * M
    dq = dscore @ kp + into * (do @ before[:, :, :, None].transpose(-1, -2))
    own_grad = ((qp * into).transpose(-1, -2) @ do).sum(3)
    after = (carry.transpose(-1, -2) @ own_grad.flatten(-2)).view_as(own_grad)
    if s["dlast"] is not None:
        rest = _powers(ld, s["lens"][:, None] - end)
        after = after + rest[..., None, None] * s["dlast"][:, :, None]
    dk = (dscore.transpose(-1, -2) @ qp).sum(3) + (out_of * (vp @ after[:, :, :, None].transpose(
        -1, -2)))[:, :, :, 0]
    dv = (score.transpose(-1, -2) @ do).sum(3) + (out_of * (kp @ after[:, :, :, None]))[:, :, :, 0]
    grads = (packed(dq * scale, q.dtype), packed(dk[:, :, :, None], k.dtype),
             packed(dv[:, :, :, None], v.dtype))
    if s["state"] is None:
        return (o,) + grads
    dstate = (own_grad * start[..., None, None]).sum(2) + whole[..., None, None] * s["dlast"]
    return (o,) + grads + (dstate,)


def _linear_step(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, Hq, D = q.shape
    Hk = k.shape[1]
    old = s["state"] * torch.exp(s["log_decay"])[:, None, None]
    if s["reset"] is not None:
        old = old.masked_fill(s["reset"][:, None, None, None], 0.0)
    new = old + k.float()[..., :, None] * v.float()[..., None, :]
    o = (q.float().view(B, Hk, Hq // Hk, D) * D ** -0.5) @ new
    return o.view(B, Hq, D).to(q.dtype), new


def _zero(t, mask):
    return t if mask is None else t * mask


def _policy(s, train):
    case, x, mask = s["case"], s["logits"].float(), s["mask"]
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(1, keepdim=True)
    a = s["actions"].long()[:, None]
    # differences of log probabilities cancel: these few numbers in 64 bits
    logp = (x.gather(1, a).double() - m.double() - z.double().log())[:, 0]
    p = e / z
    shifted = torch.where(e > 0, x - m, 0.0) - z.log()  # log p, and 0 where p is
    shifted = torch.where(e > 0, shifted, 0.0)
    entropy = -(p * shifted).sum(1)
    adv = s["advantages"].double()
    ratio = torch.exp(logp - s["old_logp"].double())
    plain, clipped = ratio * adv, ratio.clamp(1.0 - CLIP, 1.0 + CLIP) * adv
    loss = -torch.minimum(plain, clipped) - case["entropy"] * entropy.double()
    slope = torch.where(plain <= clipped, -plain, 0.0)
    outs = []
    if s["ref_logp"] is not None:
        d = s["ref_logp"].double() - logp
        kl = torch.exp(d) - d - 1.0
        loss = loss + case["kl"] * kl
        slope = slope + case["kl"] * (1.0 - torch.exp(d))
        outs = [_zero(kl.float(), mask)]
    outs = [_zero(t.float(), mask) for t in (loss, logp, entropy)] + outs
    if not train:
        return tuple(outs)
    w = _zero(s["dloss"], mask)[:, None]
    g = slope.float()[:, None]
    dx = -g * p
    if case["entropy"]:
        dx = dx + case["entropy"] * p * (shifted + entropy[:, None])
    dx.scatter_add_(1, a, g)
    return tuple(outs) + ((w * dx).to(s["logits"].dtype),)


def _distill(s, train):
    case, mask, T = s["case"], s["mask"], s["case"]["temperature"]
    x = s["logits"].float() / T
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(1, keepdim=True)
    there = s["top_ids"] >= 0
    ids = s["top_ids"].long().clamp(min=0)
    t = (s["top_logits"].double() / T).masked_fill(~there, -math.inf)
    lse = (torch.logsumexp(t, 1) if s["teacher_lse"] is None else s["teacher_lse"].double())
    logq = torch.where(there, t - lse[:, None], 0.0)
    q = torch.where(there, torch.exp(logq), 0.0)
    logp = x.gather(1, ids).double() - m.double() - z.double().log()
    loss = _zero((q * (logq - logp)).sum(1).float(), mask)
    if not train:
        return loss
    w = _zero(s["dloss"], mask)[:, None] / T
    dx = (q.sum(1, keepdim=True).float() / z) * e
    dx.scatter_add_(1, ids, -q.float())
    return loss, (w * dx).to(s["logits"].dtype)


def _plain(s):
    op = s["op"]
    if op == "linear_step":
        return _linear_step(s)
    if op.startswith("linear"):
        return _linear(s, op == "linear_train")
    return (_policy if op.startswith("policy") else _distill)(s, op.endswith("train"))


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _framework(s):
    import linear_recurrence_scan_affine_gb300 as rl
    op, case = s["op"], s["case"]
    if op == "linear_step":
        return rl.rlcs_linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"],
                                             reset=s["reset"])
    if op == "linear_prompt":
        return rl.rlcs_linear_attention(s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"],
                                        state=s["state"], return_state=True)
    if op == "linear_train":
        args = (s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"])
        out = rl.rlcs_linear_attention(*args, state=s["state"])
        dq, dk, dv, dstate = rl.rlcs_linear_attention_backward(s["dout"], *args, state=s["state"],
                                                               dlast=s["dlast"])
        return (out, dq, dk, dv) if s["state"] is None else (out, dq, dk, dv, dstate)
    if op.startswith("policy"):
        args = (s["logits"], s["actions"], s["old_logp"], s["advantages"])
        kw = dict(ref_logp=s["ref_logp"], mask=s["mask"], clip_low=CLIP, clip_high=CLIP,
                  kl_coef=case["kl"], entropy_coef=case["entropy"])
        if op == "policy_eval":
            got, dlogits = rl.rlcs_policy_loss(*args, **kw), ()
        else:  # the losses and their gradient from one reading of the logits
            dlogits, got = rl.rlcs_policy_loss_backward(s["dloss"], *args, return_loss=True, **kw)
            dlogits = (dlogits,)
        return tuple(t for t in got if t is not None) + dlogits
    args = (s["logits"], s["top_ids"], s["top_logits"])
    kw = dict(teacher_lse=s["teacher_lse"], mask=s["mask"], temperature=case["temperature"])
    if op == "distill_eval":
        return rl.rlcs_distill_loss(*args, **kw)
    dlogits, loss = rl.rlcs_distill_loss_backward(s["dloss"], *args, return_loss=True, **kw)
    return loss, dlogits


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# Work of one pass
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "linear_step":
        B, Hq, Hk, D = (case[k] for k in ("B", "Hq", "Hk", "D"))
        return {"bytes": B * (8 * Hk * D * D + 2 * D * (2 * Hq + 2 * Hk)),
                "flops": B * D * D * (4 * Hk + 2 * Hq)}
    if op.startswith("linear"):
        Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
        n = sum(_lengths(case))
        # the recurrence itself: a state's update and its product with each query
        states = 4 * case["nseq"] * Hk * D * D
        given = states if case["state"] else 0
        forward = {"bytes": 2 * n * D * (2 * Hq + 2 * Hk) + given, "flops": 2 * n * D * D * (Hq + Hk)}
        if op == "linear_prompt":
            return {"bytes": forward["bytes"] + states, "flops": forward["flops"]}
        return {"bytes": forward["bytes"] + 2 * n * D * (3 * Hq + 4 * Hk) + 3 * given,
                "flops": forward["flops"] + 2 * n * D * D * (2 * Hq + 3 * Hk)}
    n, V, e = case["tokens"], case["V"], 4 if case["dtype"] == "f32" else 2
    read = int(n * (1.0 - case["p_mask"])) * V * e + (n if case["p_mask"] else 0)
    written = n * V * e + 4 * n if op.endswith("train") else 0
    if op.startswith("policy"):
        return {"bytes": read + written + 4 * n * (8 if case["kl"] else 6),
                "flops": n * V * (10 if op.endswith("train") else 6)}
    return {"bytes": read + written + 8 * n * case["K"] + 4 * n,
            "flops": n * V * (7 if op.endswith("train") else 4)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, step by step and row by row
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("linear"):
        return _exact_step(s) if op == "linear_step" else _exact_linear(s, op == "linear_train")
    rows, train = max(1, (1 << 25) // case["V"]), op.endswith("train")
    parts = []
    for lo in range(0, case["tokens"], rows):
        at = {k: (t[lo:lo + rows] if isinstance(t, torch.Tensor) else t) for k, t in s.items()}
        parts.append((_exact_policy if op.startswith("policy") else _exact_distill)(at, train))
    out = tuple(torch.cat(p) for p in zip(*parts))
    return out[0] if op == "distill_eval" else out


def _exact_step(s):
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    group = q.shape[1] // k.shape[1]
    lam = s["log_decay"].double().exp()
    new = torch.einsum("bhd,bhe->bhde", k, v)
    keep = 1.0 if s["reset"] is None else (~s["reset"]).double()[:, None, None, None]
    new += keep * lam[None, :, None, None] * s["state"].double()
    o = torch.einsum("bhd,bhde->bhe", q, new.repeat_interleave(group, 1)) / math.sqrt(q.shape[2])
    return o, new


def _exact_linear(s, train):
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    lens = s["lens"].tolist()
    order = sorted(range(len(lens)), key=lambda i: -lens[i])  # the longest sequences first
    first = s["cu_seqlens"][:-1].long()[order]
    lam = s["log_decay"].double().exp()[:, None, None]
    active = [sum(1 for m in lens if m > t) for t in range(max(lens))]
    zeros = torch.zeros(len(lens), Hk, D, D, dtype=torch.float64, device=q.device)
    S = zeros.clone() if s["state"] is None else s["state"].double()[order]
    shared = (-1, Hk, Hq // Hk, D)
    q = q.view(shared) / math.sqrt(D)
    o = torch.empty_like(q)
    do = s["dout"].double().view(shared) if train else None
    dq = torch.empty_like(q) if train else None
    for t, m in enumerate(active):
        at, now = first[:m] + t, S[:m]
        now.mul_(lam).add_(k[at][..., :, None] * v[at][..., None, :])
        o[at] = q[at] @ now
        if train:
            dq[at] = do[at] @ now.transpose(-1, -2)
    back = torch.empty(len(lens), dtype=torch.long, device=q.device)
    back[torch.tensor(order, device=q.device)] = torch.arange(len(lens), device=q.device)
    o = o.view(-1, Hq, D)
    if not train:
        return o, S[back]
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    R = zeros.clone() if s["dlast"] is None else s["dlast"].double()[order]
    for t in range(max(lens) - 1, -1, -1):
        m = active[t]
        at, now = first[:m] + t, R[:m]
        now.add_(q[at].transpose(-1, -2) @ do[at])
        dv[at] = (k[at][:, :, None] @ now)[:, :, 0]
        dk[at] = (now @ v[at][..., None])[..., 0]
        now.mul_(lam)
    dq = dq.view(-1, Hq, D) / math.sqrt(D)
    return (o, dq, dk, dv) if s["state"] is None else (o, dq, dk, dv, R[back])


def _exact_policy(s, train):
    case = s["case"]
    n = len(s["actions"])
    logall = torch.log_softmax(s["logits"].double(), 1)
    p = logall.exp()
    logp = logall[torch.arange(n, device=p.device), s["actions"].long()]
    H = -torch.where(p > 0, p * logall, 0.0).sum(1)
    A, keep = s["advantages"].double(), 1.0 if s["mask"] is None else s["mask"].double()
    r = (logp - s["old_logp"].double()).exp()
    cut = (A > 0) & (r > 1.0 + CLIP) | (A < 0) & (r < 1.0 - CLIP)
    bound = torch.where(A > 0, 1.0 + CLIP, 1.0 - CLIP)
    loss = -torch.where(cut, bound, r) * A - case["entropy"] * H
    slope = -torch.where(cut, 0.0, r) * A
    outs = [logp, H]
    if s["ref_logp"] is not None:
        d = s["ref_logp"].double() - logp
        outs.append(torch.expm1(d) - d)
        loss = loss + case["kl"] * outs[-1]
        slope = slope - case["kl"] * torch.expm1(d)
    outs = tuple(t * keep for t in [loss] + outs)
    if not train:
        return outs
    dx = -slope[:, None] * p
    dx += case["entropy"] * torch.where(p > 0, p * (logall + H[:, None]), 0.0)
    dx[torch.arange(n, device=p.device), s["actions"].long()] += slope
    return outs + ((s["dloss"].double() * keep)[:, None] * dx,)


def _exact_distill(s, train):
    T, keep = s["case"]["temperature"], 1.0 if s["mask"] is None else s["mask"].double()
    logall = torch.log_softmax(s["logits"].double() / T, 1)
    there = (s["top_ids"] >= 0).double()
    t = s["top_logits"].double() / T
    mass = (t.exp() * there).sum(1)
    if s["teacher_lse"] is not None:
        mass = s["teacher_lse"].double().exp()
    q = t.exp() * there / mass.clamp(min=1e-300)[:, None]
    ids = s["top_ids"].long().clamp(min=0)
    own_log = logall[torch.arange(len(t), device=t.device)[:, None], ids]
    loss = torch.where(q > 0, q * (q.log() - own_log), 0.0).sum(1) * keep
    if not train:
        return (loss,)
    target = torch.zeros_like(logall).scatter_add_(1, ids, q)
    dx = logall.exp() * q.sum(1, keepdim=True) - target
    return loss, (s["dloss"].double() * keep / T)[:, None] * dx
