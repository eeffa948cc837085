"""Measured calls of the logits operators around a verify round: what a
server does with the target and draft rows before the round (penalties,
biases, grammar masks, and the token history behind them), and what it takes
from them afterwards to train the drafter (a teacher's record of top logits,
and the distillation loss with its gradient).

A case is a dict of plain values.  ``run`` computes it in elementary torch
operations, or, when ``own`` is set, by the calls of this repository's
package on the same inputs.
"""

import math

import numpy as np
import torch

own = False

NEG_INF = float("-inf")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request, one token, no drafts: the smallest call, where latency counts
        dict(name="adjust_token_f32", op="adjust", B=1, n=1, pos0=0, V=32000, dtype="f32", slots=1,
             used=200, bias=0, mask="none", inplace=False),
        # the drafter's fourth position of 16 requests, rows of odd length behind one another
        dict(name="adjust_draft_odd_bf16", op="adjust", B=16, n=1, pos0=3, V=50257, dtype="bf16",
             slots=24, used=700, bias=12, mask="loose", inplace=False),
        # the serving batch's target rows: 64 requests, 5 drafts, long answers behind them
        dict(name="adjust_round_bf16", op="adjust", B=64, n=6, pos0=0, V=128256, dtype="bf16", slots=64,
             used=1500, bias=32, mask="loose", inplace=False),
        # constrained output: a grammar that leaves few tokens, written over the rows themselves
        dict(name="grammar_round_bf16", op="adjust", B=32, n=6, pos0=0, V=152064, dtype="bf16", slots=0,
             used=0, bias=0, mask="tight", inplace=True),
        # a short prompt enters a slot
        dict(name="history_admit_one", op="history", B=1, T=33, G=5, V=32000, slots=4),
        # a batch of resumed requests: long prompts and what they had generated
        dict(name="history_admit_batch", op="history", B=64, T=4000, G=1000, V=128256, slots=64),
        # a teacher's record of one request's round, for logging
        dict(name="top_round_one_f32", op="top", B=1, n=5, V=32000, dtype="f32", K=16, temperature=1.0),
        # the serving batch's target rows turned into a teacher's record
        dict(name="top_round_bf16", op="top", B=64, n=6, V=128256, dtype="bf16", K=64, temperature=1.0),
        # held-out loss of a drafter in float32, odd vocabulary
        dict(name="loss_heldout_f32", op="loss", B=4, n=31, V=50257, dtype="f32", K=32, temperature=2.0,
             tail="renorm"),
        # the backward half of a training step of its own
        dict(name="grad_step_bf16", op="grad", B=16, n=64, V=32000, dtype="bf16", K=100, temperature=1.0,
             tail="renorm"),
        # online alignment: the draft rows of the serving batch against the round's record
        dict(name="train_online_bf16", op="loss_grad", B=64, n=5, V=128256, dtype="bf16", K=64,
             temperature=1.0, tail="bucket"),
        # a drafter's training batch: 8 sequences of 256 positions
        dict(name="train_batch_bf16", op="loss_grad", B=8, n=256, V=128256, dtype="bf16", K=64,
             temperature=1.0, tail="bucket"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["adjust", "adjust", "history", "top", "top", "loss", "grad", "loss_grad", "loss_grad"])
    V = _log_int(rng, 1000, 160000)
    if rng.random() < 0.3:
        V = rng.choice([32000, 128256, 152064])
    if op == "history":
        return dict(op=op, B=_log_int(rng, 1, 64), T=_log_int(rng, 1, 4000), G=_log_int(rng, 1, 1000), V=V,
                    slots=64 + rng.randrange(32))
    dtype = rng.choice(["f32", "bf16", "bf16"])
    if op == "adjust":
        n = _log_int(rng, 1, 9)
        B = _log_int(rng, 1, max(1, min(256, 40_000_000 // (n * V))))
        form = rng.choice(["penalties", "mask", "both", "all", "inplace"])
        if form == "inplace":
            return dict(op=op, B=B, n=n, pos0=0, V=V, dtype=dtype, slots=0, used=0, bias=0,
                        mask=rng.choice(["tight", "loose"]), inplace=True)
        pen = form != "mask"
        return dict(op=op, B=B, n=n, pos0=rng.choice([0, 0, rng.randrange(8)]), V=V, dtype=dtype,
                    slots=B + rng.randrange(9) if pen else 0,
                    used=min(_log_int(rng, 1, 4000), V) if pen else 0,
                    bias=_log_int(rng, 1, 300) if form == "all" else 0,
                    mask="none" if form == "penalties" else rng.choice(["tight", "loose"]), inplace=False)
    K = min(_log_int(rng, 1, 256), V // 2)
    T = rng.choice([1.0, 1.0, 0.7, 2.0, 4.0])
    if op == "top":
        n = _log_int(rng, 1, 9)
        B = _log_int(rng, 1, max(1, min(256, 40_000_000 // (n * V))))
        return dict(op=op, B=B, n=n, V=V, dtype=dtype, K=K, temperature=T)
    n = _log_int(rng, 1, 256)
    B = _log_int(rng, 1, max(1, min(64, 120_000_000 // (n * V))))
    return dict(op=op, B=B, n=n, V=V, dtype=dtype, K=K, temperature=T, tail=rng.choice(["bucket", "renorm"]))


# ----------------------------------------------------------------- inputs
def _rows(g, shape, sigma, boost):
    """Logits rows as a language model gives them: a normal bulk and, in every
    row, 20 likely tokens 8 above it."""
    z = torch.randn(shape, generator=g, device="cuda") * sigma
    if boost:
        idx = torch.randint(0, shape[-1], (*shape[:-1], min(20, shape[-1])), generator=g, device="cuda")
        z.scatter_add_(-1, idx, torch.full(idx.shape, 8.0, device="cuda"))
    return z


def _pack_bits(allowed):
    """Truth values [..., V] as bits of int32 words [..., ceil(V/32)], token v
    at bit v % 32 of word v // 32."""
    V = allowed.shape[-1]
    W = (V + 31) // 32
    out = torch.zeros(*allowed.shape[:-1], W, dtype=torch.int64, device=allowed.device)
    pad = torch.zeros(*allowed.shape[:-1], W * 32, dtype=torch.bool, device=allowed.device)
    pad[..., :V] = allowed
    pad = pad.view(*allowed.shape[:-1], W, 32)
    for b in range(32):
        out |= pad[..., b].to(torch.int64) << b
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def _adjust_inputs(c, g):
    B, n, V = c["B"], c["n"], c["V"]
    s = {"logits": _rows(g, (B, n, V), 3.0, True).to(DTYPES[c["dtype"]])}
    p_end = c["pos0"] + n - 1
    s["drafts"] = torch.randint(0, V, (B, max(p_end, 1)), generator=g, device="cuda", dtype=torch.int32)
    if c["slots"]:
        S, U = c["slots"], c["used"]
        s["slot"] = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
        s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device="cuda")
        s["presence"] = torch.rand(B, generator=g, device="cuda")
        s["frequency"] = 0.5 * torch.rand(B, generator=g, device="cuda")
        # tokens used so far: skewed to low ids, a part of them in the prompt only
        u = torch.rand(S, U, generator=g, device="cuda")
        tok = (u * u * V).long().clamp_(max=V - 1)
        counts = torch.zeros(S, V, dtype=torch.int32, device="cuda")
        half = U // 2
        counts.scatter_add_(1, tok[:, half:], torch.ones(S, U - half, dtype=torch.int32, device="cuda"))
        seen = torch.zeros(S, V, dtype=torch.bool, device="cuda")
        seen.scatter_(1, tok, True)
        s["counts"], s["seen"] = counts, _pack_bits(seen)
    if c["bias"]:
        nb = torch.randint(0, c["bias"] + 1, (B,), generator=g, device="cuda")
        off = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        off[1:] = nb.cumsum(0).to(torch.int32)
        total = int(off[-1])
        s["bias_offsets"] = off
        s["bias_tokens"] = torch.randint(0, V, (total,), generator=g, device="cuda", dtype=torch.int32)
        s["bias_values"] = 4.0 * torch.randn(total, generator=g, device="cuda")
    if c["mask"] != "none":
        if c["mask"] == "tight":
            allowed = torch.zeros(B, n, V, dtype=torch.bool, device="cuda")
            idx = torch.randint(0, V, (B, n, 64), generator=g, device="cuda")
            allowed.scatter_(-1, idx, True)
        else:
            allowed = torch.rand(B, n, V, generator=g, device="cuda") < 0.9
        s["mask"] = _pack_bits(allowed)
    return s


def _history_inputs(c, g):
    B, T, G, V, S = c["B"], c["T"], c["G"], c["V"], c["slots"]
    s = {}
    for name, width in (("prompt", T), ("generated", G)):
        u = torch.rand(B, width, generator=g, device="cuda")
        s[name] = (u * u * V).to(torch.int32).clamp_(max=V - 1)
        s[name + "_len"] = torch.randint((width + 1) // 2, width + 1, (B,), generator=g, device="cuda",
                                         dtype=torch.int32)
    s["slot"] = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
    # what earlier requests left in the slots
    u = torch.rand(S, 500, generator=g, device="cuda")
    tok = (u * u * V).long().clamp_(max=V - 1)
    s["counts"] = torch.zeros(S, V, dtype=torch.int32, device="cuda").scatter_add_(
        1, tok[:, :250], torch.ones(S, 250, dtype=torch.int32, device="cuda"))
    s["seen"] = _pack_bits(torch.zeros(S, V, dtype=torch.bool, device="cuda").scatter_(1, tok, True))
    return s


def _distill_inputs(c, g):
    B, n, V, K, T = c["B"], c["n"], c["V"], c["K"], c["temperature"]
    s = {"student": torch.empty(B, n, V, dtype=DTYPES[c["dtype"]], device="cuda"),
         "tokens": torch.empty(B, n, K, dtype=torch.int32, device="cuda"),
         "logits": torch.empty(B, n, K, device="cuda"),
         "lse": torch.empty(B, n, 2, device="cuda")}
    student, tokens, logits, lse = (s[k].view(B * n, -1) for k in ("student", "tokens", "logits", "lse"))
    step = max(1, 32_000_000 // V)
    for r in range(0, B * n, step):
        e = min(r + step, B * n)
        z = _rows(g, (e - r, V), 3.0, True)
        val, idx = z.topk(K, dim=-1)
        tokens[r:e], logits[r:e] = idx.to(torch.int32), val
        x = z / T
        lse[r:e, 0] = torch.logsumexp(x, -1)
        lse[r:e, 1] = torch.logsumexp(x.scatter_(-1, idx, NEG_INF), -1)
        z += torch.randn(z.shape, generator=g, device="cuda")
        student[r:e] = z.to(student.dtype)
    # positions of the prompt carry no loss
    keep = (torch.rand(B, n, generator=g, device="cuda") < 0.9).float()
    s["weights"] = keep / keep.sum().clamp(min=1.0)
    if c["op"] == "grad":
        for r in range(0, B * n, step):
            e = min(r + step, B * n)
            x = student[r:e].double() / T
            s.setdefault("student_lse", torch.empty(B, n, 2, device="cuda"))
            sl = s["student_lse"].view(B * n, 2)
            sl[r:e, 0] = torch.logsumexp(x, -1)
            sl[r:e, 1] = torch.logsumexp(x.scatter(-1, tokens[r:e].long(), NEG_INF), -1)
    return s


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "adjust":
        return _adjust_inputs(c, g)
    if c["op"] == "history":
        return _history_inputs(c, g)
    if c["op"] == "top":
        return {"teacher": _rows(g, (c["B"], c["n"], c["V"]), 3.0, True).to(DTYPES[c["dtype"]])}
    return _distill_inputs(c, g)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        # the handle, records and output buffers that a serving or training program keeps
        import speculative_decoding_verification_sampling_amd as sv
        c = case
        s["v"] = sv.Verifier(min(c["B"], 64), 5, c["V"])
        if c["op"] == "adjust":
            s["out"] = s["logits"] if c["inplace"] else torch.empty_like(s["logits"])
            if c["slots"]:
                s["history"] = sv.TokenHistory(c["slots"], c["V"], counts=s["counts"], seen=s["seen"])
                s["penalties"] = sv.make_penalties(c["B"], s["repetition"].tolist(), s["presence"].tolist(),
                                                   s["frequency"].tolist(), s["slot"].tolist())
        elif c["op"] == "history":
            s["history"] = sv.TokenHistory(c["slots"], c["V"], counts=s["counts"], seen=s["seen"])
        elif c["op"] in ("grad", "loss_grad"):
            s["grad"] = torch.empty_like(s["student"])
    return s


# -------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if own:
        return {"adjust": _own_adjust, "history": _own_history, "top": _own_top}.get(op, _own_distill)(state)
    return {"adjust": _plain_adjust, "history": _plain_history, "top": _plain_top}.get(op, _plain_distill)(state)


def _own_adjust(s):
    c = s["case"]
    bias = (s["bias_offsets"], s["bias_tokens"], s["bias_values"]) if c["bias"] else None
    return s["v"].adjust_logits(s["logits"], penalties=s.get("penalties"), history=s.get("history"),
                                draft_tokens=s["drafts"] if c["slots"] else None, pos0=c["pos0"], bias=bias,
                                mask=s.get("mask"), out=s["out"])


def _own_history(s):
    h = s["history"]
    s["v"].history_reset(h, s["slot"])
    s["v"].history_add(h, s["slot"], s["prompt"], s["prompt_len"], prompt=True)
    s["v"].history_add(h, s["slot"], s["generated"], s["generated_len"])
    return h.counts, h.seen


def _own_top(s):
    c = s["case"]
    r = s["v"].top_logits(s["teacher"], c["K"], temperature=c["temperature"])
    return r["tokens"], r["logits"], r["lse"]


def _own_distill(s):
    c = s["case"]
    rec = {"tokens": s["tokens"], "logits": s["logits"], "lse": s["lse"]}
    kw = dict(weights=s["weights"], temperature=c["temperature"], tail=c["tail"])
    if c["op"] == "loss":
        o = s["v"].distill_loss(s["student"], rec, **kw)
        return o["loss"], o["lse"]
    if c["op"] == "grad":
        return s["v"].distill_grad(s["student"], rec, s["student_lse"], grad=s["grad"], **kw)
    o = s["v"].distill_loss_grad(s["student"], rec, grad=s["grad"], **kw)
    return o["loss"], o["grad"]


def _unpack_bits(words, V):
    bit = torch.arange(32, device=words.device, dtype=torch.int32)
    return ((words.unsqueeze(-1) >> bit) & 1).flatten(-2)[..., :V].bool()


def _plain_adjust(s):
    c = s["case"]
    B, n, V = c["B"], c["n"], c["V"]
    z = s["logits"].float()
    if c["slots"]:
        slot = s["slot"].long()
        count = s["counts"][slot].unsqueeze(1).repeat(1, n, 1)
        seen = _unpack_bits(s["seen"][slot], V).unsqueeze(1).repeat(1, n, 1)
        for i in range(n):
            before = s["drafts"][:, :c["pos0"] + i].long()
            count[:, i].scatter_add_(1, before, torch.ones_like(before, dtype=torch.int32))
            seen[:, i].scatter_(1, before, True)
        r = s["repetition"].view(B, 1, 1)
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        used = z - s["frequency"].view(B, 1, 1) * count.float() - s["presence"].view(B, 1, 1)
        z = torch.where(count > 0, used, z)
    if c["bias"]:
        row = torch.repeat_interleave(torch.arange(B, device=z.device), s["bias_offsets"].diff().long(),
                                      output_size=s["bias_tokens"].numel())
        bias = torch.zeros(B, V, device=z.device)
        bias.index_put_((row, s["bias_tokens"].long()), s["bias_values"], accumulate=True)
        z = z + bias.unsqueeze(1)
    if c["mask"] != "none":
        z = z.masked_fill(~_unpack_bits(s["mask"], V), NEG_INF)
    z = z.to(s["logits"].dtype)
    return s["logits"].copy_(z) if c["inplace"] else z


def _plain_history(s):
    V, slot = s["case"]["V"], s["slot"].long()
    counts, words = s["counts"], s["seen"]
    seen = torch.zeros(len(slot), V + 1, dtype=torch.bool, device=counts.device)
    fresh = torch.zeros(len(slot), V + 1, dtype=torch.int32, device=counts.device)
    for name in ("prompt", "generated"):
        tok = s[name].long()
        valid = torch.arange(tok.shape[1], device=tok.device) < s[name + "_len"].unsqueeze(1)
        tok = torch.where(valid, tok, V)
        seen.scatter_(1, tok, True)
        if name == "generated":
            fresh.scatter_add_(1, tok, torch.ones_like(tok, dtype=torch.int32))
    counts[slot] = fresh[:, :V]
    words[slot] = _pack_bits(seen[:, :V])
    return counts, words


def _plain_top(s):
    c = s["case"]
    z = s["teacher"].float()
    # ties go to the lowest index: a stable order
    val, idx = torch.sort(z, dim=-1, descending=True, stable=True)
    K, T = c["K"], c["temperature"]
    x = val / T
    m = x[..., :1]
    rest_m = x[..., K:K + 1]
    rest = (x[..., K:] - rest_m).exp().sum(-1, keepdim=True)
    total = (x - m).exp().sum(-1, keepdim=True)
    lse = torch.cat([m + total.log(), rest_m + rest.log()], -1)
    return idx[..., :K].to(torch.int32), val[..., :K].contiguous(), lse


def _plain_distill(s):
    c = s["case"]
    T, bucket = c["temperature"], c["tail"] == "bucket"
    x = s["student"].float() / T
    idx = s["tokens"].long()
    t = s["logits"] / T
    w = s["weights"].unsqueeze(-1)
    if bucket:
        logp = t - s["lse"][..., :1]
        logp_rest = s["lse"][..., 1:] - s["lse"][..., :1]
    else:
        mt = t.amax(-1, keepdim=True)
        logp = t - mt - (t - mt).exp().sum(-1, keepdim=True).log()
    p = logp.exp()
    sel = x.gather(-1, idx)
    if c["op"] == "grad":
        lse, rest_lse = s["student_lse"][..., :1], s["student_lse"][..., 1:]
    else:
        m = x.amax(-1, keepdim=True)
        lse = m + (x - m).exp().sum(-1, keepdim=True).log()
        rest = x.scatter(-1, idx, NEG_INF)
        rm = rest.amax(-1, keepdim=True)
        rest_lse = rm + (rest - rm).exp().sum(-1, keepdim=True).log()
        loss = (p * (logp - (sel - lse))).sum(-1, keepdim=True)
        if bucket:
            loss = loss + logp_rest.exp() * (logp_rest - (rest_lse - lse))
        loss = (loss * w).squeeze(-1)
        if c["op"] == "loss":
            return loss, torch.cat([lse, rest_lse], -1)
    P = p.sum(-1, keepdim=True)
    if bucket:
        P = P + logp_rest.exp()
    q_sel = (sel - lse).exp() * P - p
    if bucket:
        grad = (x - lse).exp_().mul_(P).sub_((x - rest_lse).exp_().mul_(logp_rest.exp()))
    else:
        grad = (x - lse).exp_().mul_(P)
    grad.scatter_(-1, idx, q_sel)
    grad = (grad * (w / T)).to(s["student"].dtype)
    if c["op"] == "grad":
        return grad
    return loss, grad


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "adjust":
        return _exact_adjust(case, s)
    if op == "history":
        return _exact_history(case, s)
    if op == "top":
        return _exact_top(case, s)
    return _exact_distill(case, s)


def _exact_adjust(c, s):
    """Row by row: only the tokens that a rule names are touched."""
    B, n, V = c["B"], c["n"], c["V"]
    z = s["logits"].double()
    for b in range(B):
        base = {}
        if c["slots"]:
            k = int(s["slot"][b])
            bits = np.unpackbits(s["seen"][k].cpu().numpy().view(np.uint8), bitorder="little")[:V]
            cnt = s["counts"][k].cpu().numpy()
            base = {int(t): int(cnt[t]) for t in np.nonzero(bits)[0]}
            rep, pres, freq = (float(s[x][b]) for x in ("repetition", "presence", "frequency"))
        bias = {}
        if c["bias"]:
            lo, hi = int(s["bias_offsets"][b]), int(s["bias_offsets"][b + 1])
            for t, v in zip(s["bias_tokens"][lo:hi].tolist(), s["bias_values"][lo:hi].tolist()):
                bias[t] = bias.get(t, 0.0) + v
        for i in range(n):
            row = z[b, i]
            if c["slots"]:
                use = dict(base)
                for t in s["drafts"][b, :c["pos0"] + i].tolist():
                    use[t] = use.get(t, 0) + 1
                idx = torch.tensor(list(use), dtype=torch.long, device=z.device)
                num = torch.tensor(list(use.values()), dtype=torch.float64, device=z.device)
                x = row[idx]
                x = torch.where(x > 0, x / rep, x * rep)
                row[idx] = x - torch.where(num > 0, freq * num + pres, 0.0)
            if bias:
                row[torch.tensor(list(bias), dtype=torch.long, device=z.device)] += torch.tensor(
                    list(bias.values()), dtype=torch.float64, device=z.device)
            if c["mask"] != "none":
                bits = np.unpackbits(s["mask"][b, i].cpu().numpy().view(np.uint8), bitorder="little")[:V]
                row[torch.from_numpy(bits == 0).to(z.device)] = NEG_INF
    return z


def _exact_history(c, s):
    V = c["V"]
    counts, words = s["counts"].cpu().numpy().copy(), s["seen"].cpu().numpy().copy()
    W = words.shape[1]
    for b, k in enumerate(s["slot"].tolist()):
        prompt = s["prompt"][b, :int(s["prompt_len"][b])].cpu().numpy()
        gen = s["generated"][b, :int(s["generated_len"][b])].cpu().numpy()
        counts[k] = np.bincount(gen, minlength=V)
        bits = np.zeros(W * 32, np.uint8)
        bits[prompt] = 1
        bits[gen] = 1
        words[k] = np.packbits(bits, bitorder="little").view(np.int32)
    return torch.from_numpy(counts), torch.from_numpy(words)


def _exact_top(c, s):
    B, n, K, T = c["B"], c["n"], c["K"], c["temperature"]
    tokens = np.empty((B, n, K), np.int32)
    logits = np.empty((B, n, K))
    lse = np.empty((B, n, 2))
    for b in range(B):
        for i in range(n):
            z = s["teacher"][b, i].double().cpu().numpy()
            cand = np.nonzero(z >= np.partition(z, -K)[-K])[0]
            top = cand[np.lexsort((cand, -z[cand]))][:K]
            tokens[b, i], logits[b, i] = top, z[top]
            e = np.exp((z - z.max()) / T)
            lse[b, i, 0] = z.max() / T + math.log(e.sum())
            z[top] = NEG_INF
            lse[b, i, 1] = z.max() / T + math.log(np.exp((z - z.max()) / T).sum())
    return torch.from_numpy(tokens), torch.from_numpy(logits), torch.from_numpy(lse)


def _exact_distill(c, s):
    """Row blocks in float64, the gradient from the two softmaxes (the whole
    row's and the rest's) rather than from their logarithms."""
    B, n, V, T = c["B"], c["n"], c["V"], c["temperature"]
    R = B * n
    bucket = c["tail"] == "bucket"
    student = s["student"].view(R, V)
    idx = s["tokens"].view(R, -1).long()
    t = s["logits"].view(R, -1).double()
    tl = s["lse"].view(R, 2).double()
    w = s["weights"].view(R).double()
    loss = torch.empty(R, dtype=torch.float64, device=student.device)
    lse = torch.empty(R, 2, dtype=torch.float64, device=student.device)
    grad = torch.empty(R, V, dtype=torch.float64) if c["op"] != "loss" else None
    step = max(1, 16_000_000 // V)
    for r in range(0, R, step):
        e = min(r + step, R)
        x = student[r:e].double() / T
        inside = torch.zeros(x.shape, dtype=torch.bool, device=x.device).scatter_(1, idx[r:e], True)
        lse[r:e, 0] = torch.logsumexp(x, 1)
        lse[r:e, 1] = torch.logsumexp(x.masked_fill(inside, NEG_INF), 1)
        if bucket:
            p = torch.exp(t[r:e] / T - tl[r:e, :1])
            p_rest = torch.exp(tl[r:e, 1] - tl[r:e, 0])
        else:
            p = torch.softmax(t[r:e] / T, 1)
            p_rest = torch.zeros(e - r, dtype=torch.float64, device=x.device)
        sl = lse[r:e]
        if c["op"] == "grad":
            sl = s["student_lse"].view(R, 2)[r:e].double()
        logq = x.gather(1, idx[r:e]) - sl[:, :1]
        kl = (p * (p.log() - logq)).sum(1)
        if bucket:
            kl = kl + p_rest * (p_rest.log() - (sl[:, 1] - sl[:, 0]))
        loss[r:e] = w[r:e] * kl
        if grad is not None:
            q = torch.exp(x - sl[:, :1])
            d = q * (p.sum(1) + p_rest).unsqueeze(1)
            d.scatter_add_(1, idx[r:e], -p)
            if bucket:
                d -= p_rest.unsqueeze(1) * torch.exp(x - sl[:, 1:]).masked_fill(inside, 0.0)
            grad[r:e] = (d * (w[r:e] / T).unsqueeze(1)).cpu()
    if c["op"] == "loss":
        return loss.view(B, n), lse.view(B, n, 2)
    if c["op"] == "grad":
        return grad.view(B, n, V)
    return loss.view(B, n), grad.view(B, n, V)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    V = c["V"]
    if c["op"] == "history":
        tokens = c["B"] * (c["T"] + c["G"]) * 3 // 4        # a half to all of each row is valid
        # token ids; the seen words of the slots; the counts that are touched
        return {"bytes": 4 * tokens + 8 * c["B"] * ((V + 31) // 32) + 8 * c["B"] * c["G"] * 3 // 4,
                "flops": tokens}
    es = 4 if c["dtype"] == "f32" else 2
    rows = c["B"] * c["n"]
    if c["op"] == "adjust":
        words = (V + 31) // 32 * 4
        share = {"none": 1.0, "loose": 1.0, "tight": 64 / V}[c["mask"]]     # logits that have to be read
        read = int(rows * V * es * share) if not c["inplace"] else 0
        masks = rows * words if c["mask"] != "none" else 0
        hist = c["B"] * (words + 4 * min(c["used"], V)) if c["slots"] else 0
        wrote = rows * V * es
        if c["inplace"] and c["mask"] == "loose":
            wrote = wrote // 10
        return {"bytes": read + wrote + masks + hist + 8 * c["B"] * c["bias"] // 2, "flops": 2 * rows * V}
    if c["op"] == "top":
        return {"bytes": rows * (V * es + 8 * c["K"] + 8), "flops": 4 * rows * V}
    record = rows * (8 * c["K"] + 12)
    if c["op"] == "loss":
        return {"bytes": rows * V * es + record + 12 * rows, "flops": 4 * rows * V}
    if c["op"] == "grad":
        return {"bytes": 2 * rows * V * es + record + 8 * rows, "flops": 4 * rows * V}
    return {"bytes": 2 * rows * V * es + record + 4 * rows, "flops": 8 * rows * V}
