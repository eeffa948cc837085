"""specv_distill_* against the float64 oracle.

Tolerances.  E = (V / 256 + 40 + 6 (1 + |L| + |max| / T)) 2^-24 bounds a
log-sum-exp (see test_gpu_record.py).  A probability exp(a - b) taken in
float32 is off by d(a) = (8 + 4 |a - b| + |a| + |b|) 2^-24 relative, plus its
log-sum-exp's E.  With those, a loss is off by at most
  w * (sum_j p_j (d_j |log p_j - log q_j| + d_j + E + (K + 40) 2^-24 |...|))
and a gradient by half a step of its type and
  w / T * (P q d + p d + p_o r d),  r = q_v / q_o outside S.
"""

import numpy as np
import pytest
import torch

from oracle import logits as ol
import speculative_decoding_verification_sampling_amd as sv

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    sv.load_library()
    return torch.device("cuda:0")


def _record(teacher, K, T):
    """The oracle's record of rows [B, n, V] as float32 tensors."""
    B, n, V = teacher.shape
    tok, val, lse = np.empty((B, n, K), np.int32), np.empty((B, n, K), np.float32), np.empty((B, n, 2), np.float32)
    for b in range(B):
        for i in range(n):
            t, x, a, o = ol.top_logits(teacher[b, i].double().numpy(), K, T)
            tok[b, i], val[b, i], lse[b, i] = t, x, (a, o)
    return {"tokens": torch.from_numpy(tok), "logits": torch.from_numpy(val), "lse": torch.from_numpy(lse)}


def _check_row(z, tok, val, tl, w, T, tail, u, loss, lse, grad, flag, skip_zero):
    V, K = len(z), len(tok)
    want, wgrad, (L, Lo), ok = ol.distill(z, tok, val, tl, T, tail, w)
    if w == 0:
        if loss is not None:
            assert loss == 0
        if grad is not None:
            assert not grad.any()
        if skip_zero:
            assert flag == 0
            return
    elif flag is not None:
        assert flag == (0 if ok else sv.FLAG_NONFINITE_ROW)
    if not ol.usable(z):
        if lse is not None:
            assert np.isnan(lse).all()
    amax = np.abs(z[np.isfinite(z)]).max() / T if np.isfinite(z).any() else 0.0
    E = lambda x: (V / 256 + 40 + 6 * (1 + abs(x) + amax)) * U
    if lse is not None and ol.usable(z):
        for g, x in zip(lse, (L, Lo)):
            assert (g == x) if not np.isfinite(x) else abs(g - x) <= E(x), (g, x)
    pr = ol.teacher_probs(tok, val, tl, V, T, tail)
    if w == 0 or pr is None or not ol.usable(z):
        if loss is not None:
            assert np.array_equal(loss, want, equal_nan=True)
        if grad is not None:
            assert np.array_equal(grad, wgrad, equal_nan=True)
        return
    p, p_rest = pr
    x = z / T
    # the log-sum-exp that the teacher's probabilities were taken with: the record's, or its own over the record
    live = (tok >= 0) & (tok < V)
    A = abs(tl[0]) if tail == "bucket" else abs(ol.log_sum_exp(val[live] / T))
    if loss is not None:
        if not np.isfinite(want):
            assert loss == want
        else:
            err = 0.0
            for t, v, pj in zip(tok, val, p):
                if pj > 0:
                    d = (8 + 4 * abs(np.log(pj)) + 2 * abs(v / T) + A + 40) * U
                    term = abs(np.log(pj) - (x[t] - L))
                    err += pj * (d * (term + 1) + E(L) + 4 * U * abs(x[t]) + (K + 40) * U * term)
            if p_rest > 0:
                d = (8 + 5 * abs(np.log(p_rest)) + A) * U
                term = abs(np.log(p_rest) - (Lo - L))
                err += p_rest * (d * (term + 1) + E(L) + E(Lo) + (K + 40) * U * term)
            assert abs(loss - want) <= w * err + 4 * U * abs(want) + 1e-38, (loss, want, w * err)
    if grad is not None:
        q = np.exp(x - L)
        with np.errstate(invalid="ignore"):
            dq = (8 + 4 * np.abs(x - L) + np.abs(x) + abs(L)) * U + E(L)
        dq = np.where(np.isfinite(dq), dq, 0.0)
        err = (p.sum() + p_rest) * q * (dq + (K + 8) * U)
        inside = np.zeros(V, bool)
        for t, v, pj in zip(tok, val, p):
            if 0 <= t < V:
                inside[t] = True
                if pj > 0:
                    err[t] += pj * (8 + 4 * abs(np.log(pj)) + 2 * abs(v / T) + A + 40 + K) * U
        if p_rest > 0 and Lo > -np.inf:
            with np.errstate(invalid="ignore"):
                r = np.where(inside, 0.0, np.exp(x - Lo))
                dr = (8 + 4 * np.abs(x - Lo) + np.abs(x) + abs(Lo)) * U + E(Lo)
            dr = np.where(np.isfinite(dr), dr, 0.0)
            err += p_rest * r * (dr + (8 + 5 * abs(np.log(p_rest)) + A) * U)
        tol = u * np.abs(wgrad) + w / T * err * 1.01 + 1e-37
        worst = np.abs(grad - wgrad) - tol
        assert (worst <= 0).all(), (int(worst.argmax()), grad[worst.argmax()], wgrad[worst.argmax()])


def _check(student, rec, weights, T, tail, out, grad, skip_zero=False):
    B, n, V = student.shape
    u = torch.finfo(student.dtype).eps / 2
    z = student.double().numpy()
    tok, val = rec["tokens"].numpy(), rec["logits"].double().numpy()
    tl = rec["lse"].double().numpy() if "lse" in rec else np.zeros((B, n, 2))
    get = lambda k: out[k].cpu().double().numpy() if out is not None and k in out else None
    loss, lse, flags = get("loss"), get("lse"), get("flags")
    g = grad.cpu().double().numpy() if grad is not None else None
    for b in range(B):
        for i in range(n):
            w = 1.0 if weights is None else float(weights[b, i])
            _check_row(z[b, i], tok[b, i], val[b, i], tl[b, i], w, T, tail, u,
                       None if loss is None else loss[b, i], None if lse is None else lse[b, i],
                       None if g is None else g[b, i], None if flags is None else int(flags[b, i]), skip_zero)


def _no_workspace(v):
    """The calls of v then take one workgroup per row."""
    v._distill_work = lambda *a: (None, 0, None)


def _run(student, rec, weights, T, tail):
    """The three calls on the same rows; all outputs checked, with and without
    a workspace (parts of rows, whole rows) where the library asks for one."""
    out = _run_form(student, rec, weights, T, tail, True)
    code = 1 if student.dtype == torch.bfloat16 else 0
    if sv.load_library().specv_distill_workspace(code, *student.shape, rec["tokens"].shape[2]) > 0:
        _run_form(student, rec, weights, T, tail, False)
    return out


def _run_form(student, rec, weights, T, tail, workspace):
    dev = {k: v.cuda() for k, v in rec.items()}
    w = None if weights is None else weights.cuda()
    kw = dict(weights=w, temperature=T, tail=tail)
    with sv.Verifier(1, 0, student.shape[2]) as v:
        if not workspace:
            _no_workspace(v)
        x = student.cuda()
        a = v.distill_loss(x, dev, **kw)
        g = v.distill_grad(x, dev, a["lse"], **kw)
        both = v.distill_loss_grad(x, dev, **kw)
        assert torch.equal(x.cpu().view(torch.uint8), student.view(torch.uint8))
        _check(student, rec, weights, T, tail, a, None)
        _check(student, rec, weights, T, tail, None, g)
        _check(student, rec, weights, T, tail, {k: both[k] for k in ("loss", "flags")}, both["grad"], True)
        y = x.clone()
        c = v.distill_loss_grad(y, dev, grad=y, **kw)
        assert c["grad"] is y
        assert torch.equal(y.view(torch.uint8), both["grad"].view(torch.uint8))
        assert torch.equal(c["loss"].view(torch.int32), both["loss"].view(torch.int32))
        y = x.clone()
        v.distill_grad(y, dev, a["lse"], grad=y, **kw)
        assert torch.equal(y.view(torch.uint8), g.view(torch.uint8))
    return a, g, both


def _rows(seed, B, n, V, dtype, noise=1.0):
    rng = np.random.default_rng(seed)
    t = rng.normal(0, 3, (B, n, V)).astype(np.float32)
    s = (t + noise * rng.normal(0, 1, t.shape)).astype(np.float32)
    return torch.from_numpy(t), torch.from_numpy(s).to(DTYPES[dtype])


@pytest.mark.parametrize("tail", ["bucket", "renorm"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,n,V,K,T", [
    (1, 1, 1, 1, 1.0), (1, 2, 2, 1, 1.0), (2, 3, 7, 3, 0.5), (2, 2, 33, 33, 2.0), (1, 2, 100, 256, 1.0),
    (3, 2, 1025, 17, 1.0), (2, 1, 8193, 256, 4.0), (2, 3, 20001, 64, 0.7), (1, 2, 50257, 32, 1.0),
    (1, 2, 128256, 64, 1.0), (1, 1, 152064, 5, 1.0), (1, 1, 200003, 64, 1.0), (1, 1, 524288, 256, 1.0)])
def test_against_the_oracle(gpu, dtype, tail, B, n, V, K, T):
    t, s = _rows(V * 3 + K, B, n, V, dtype)
    rng = np.random.default_rng(1)
    w = torch.from_numpy(rng.uniform(0.1, 2.0, (B, n)).astype(np.float32))
    if B * n > 2:
        w[0, 0] = 0.0
    _run(s, _record(t, K, T), w, T, tail)


EDGES = [4095, 4096, 4097, 8192, 8200, 16384, 16385, 32767, 32768, 32776, 32777, 49152, 49153, 65536, 65537, 73729,
         98304, 98305, 131072, 131073]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", EDGES)
def test_sizes_at_the_edges(gpu, dtype, V):
    """Lengths where groups, held groups, streamed steps and parts end."""
    t, s = _rows(V, 1, 2, V, dtype)
    rec = _record(t, 9, 1.0)
    rec["tokens"][0, 1, 0] = V - 1                                  # the last token, whatever it holds
    rec["tokens"][0, 1, 1] = 0
    _run(s, rec, None, 1.0, "bucket")


@pytest.mark.parametrize("tail", ["bucket", "renorm"])
def test_weights_left_out_and_one_row_alike(gpu, tail):
    t, s = _rows(3, 2, 3, 3001, "bf16")
    rec = _record(t, 20, 1.0)
    a, g, both = _run(s, rec, None, 1.0, tail)
    _, _, ones = _run(s, rec, torch.ones(2, 3), 1.0, tail)
    assert torch.equal(both["grad"], ones["grad"]) and torch.equal(both["loss"], ones["loss"])


@pytest.mark.parametrize("tail", ["bucket", "renorm"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [2500, 100003])
def test_records_with_gaps_and_repeats(gpu, dtype, tail, V):
    """Ignored tokens, the same token more than once, -inf logits, a record
    with one live entry."""
    B, n, K = 5, 2, 12
    t, s = _rows(17, B, n, V, dtype)
    rec = _record(t, K, 1.0)
    rec["tokens"][0, 0, 3] = -1
    rec["tokens"][0, 0, 4] = V
    rec["tokens"][0, 1, 5] = rec["tokens"][0, 1, 0]
    rec["tokens"][0, 1, 6] = rec["tokens"][0, 1, 0]
    rec["logits"][1, 0, 6:] = -float("inf")
    rec["tokens"][1, 1, 1:] = -1
    rec["tokens"][2] = rec["tokens"][2, :1, :1]                     # all entries one token
    rec["tokens"][4, 0, 1] = rec["tokens"][4, 0, 0]                 # twice, without a student's mass
    s[4, 0, rec["tokens"][4, 0, 0].item()] = -float("inf")
    _run(s, rec, None, 1.0, tail)


@pytest.mark.parametrize("tail", ["bucket", "renorm"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 9000, 140001])
def test_masked_and_broken_rows(gpu, dtype, tail, V):
    B, n, K = 10, 1, 8
    t, s = _rows(V, B, n, V, dtype)
    rec = _record(t, K, 1.0)
    inf = float("inf")
    s[0, 0, V - 1] = float("nan")
    s[1, 0, 0] = inf
    s[2] = -inf                                                     # a student row that is empty
    s[3, 0, rec["tokens"][3, 0, 0].item()] = -inf                   # no mass where the teacher has some
    inside = rec["tokens"][4, 0].long()
    keep = s[4, 0, inside].clone()
    s[4] = -inf
    s[4, 0, inside] = keep                                          # nothing outside the record
    s[5, 0, inside] = -inf
    s[6, 0, ::2] = torch.finfo(DTYPES[dtype]).min                   # masks of the type's lowest value
    rec["lse"][7] = float("nan")
    rec["logits"][8, 0, 1] = float("nan")
    rec["tokens"][9] = -1
    w = torch.ones(B, n)
    _run(s, rec, w, 1.0, tail)
    w[0:3] = 0.0                                                    # rows that carry no loss
    _run(s, rec, w, 1.0, tail)


def test_confident_student_and_teacher(gpu):
    """Rests far below the record on both sides: sums of their own."""
    V, K = 5000, 4
    t, s = _rows(23, 4, 1, V, "f32")
    t[:, :, :K] += torch.tensor([30.0, 31.0, 29.0, 28.0])
    s[0, 0, :K] += 30.0
    s[1, 0, :K] += 60.0
    s[2, 0, :K] += 150.0                                            # q_o below the smallest float
    s[3, 0, :K] -= 150.0
    for tail in ("bucket", "renorm"):
        _run(s, _record(t, K, 1.0), None, 1.0, tail)


def test_strides_and_rows_behind(gpu):
    """Rows padded, at odd addresses, position-major; nothing else written;
    a record with the bonus row behind the drafts."""
    B, n, V, K = 3, 2, 1003, 9
    t, s = _rows(29, B, n + 1, V, "bf16")
    rec = {k: x.cuda() for k, x in _record(t, K, 1.0).items()}
    s = s[:, :n].contiguous()
    short = {k: x[:, :n].contiguous() for k, x in rec.items()}
    with sv.Verifier(1, 0, V) as v:
        want = v.distill_loss_grad(s.cuda(), short)
        _check(s, {k: x.cpu() for k, x in short.items()}, None, 1.0, "bucket",
               {"loss": want["loss"], "flags": want["flags"]}, want["grad"])
        got = v.distill_loss_grad(s.cuda(), rec)
        assert torch.equal(got["grad"], want["grad"]) and torch.equal(got["loss"], want["loss"])
        for strides, off in (((n * 1024, 1024, 1), 1), ((1003, 3 * 1003, 1), 3)):
            xin = torch.as_strided(torch.zeros(B * n * 1024 + 8, dtype=torch.bfloat16, device="cuda"), (B, n, V), strides, off)
            xin.copy_(s)
            buf = torch.full((B * n * 1024 + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
            g = torch.as_strided(buf, (B, n, V), strides, off)
            o = v.distill_loss_grad(xin, rec, grad=g)
            assert torch.equal(g, want["grad"]) and torch.equal(o["loss"], want["loss"])
            outside = torch.ones_like(buf, dtype=torch.bool)
            torch.as_strided(outside, (B, n, V), strides, off).fill_(False)
            assert (buf[outside] == 7.0).all()
            a = v.distill_loss(xin, rec)
            g2 = v.distill_grad(xin, rec, a["lse"], grad=torch.as_strided(buf, (B, n, V), strides, off))
            _check(s, {k: x.cpu() for k, x in short.items()}, None, 1.0, "bucket", a, g2)
            assert (buf[outside] == 7.0).all()
        one = s[:1, :1].cuda().expand(B, n, V)                      # one student row for all
        assert torch.equal(v.distill_loss_grad(one, rec)["grad"], v.distill_loss_grad(one.contiguous(), rec)["grad"])


def test_gradient_against_differences_of_the_kernel(gpu):
    """Central differences of the kernel's own float32 loss, h = 2^-4: the
    third derivative of a log-sum-exp is below 0.2 / T^3, so the difference is
    off by h^2 / 6 * 0.2 < 1.4e-4, and by the loss's rounding
    (|loss| + |L|) * 64 * 2^-24 / h < 1e-3 at |L| < 12."""
    V, K = 50, 6
    t, s = _rows(31, 1, 1, V, "f32")
    rec = {k: x.cuda() for k, x in _record(t, K, 1.0).items()}
    h = 2.0 ** -4
    step = torch.eye(V, device="cuda") * h
    with sv.Verifier(1, 0, V) as v:
        grad = v.distill_loss_grad(s.cuda(), rec)["grad"][0, 0]
        wide = {k: x.expand(2 * V, 1, -1).contiguous() for k, x in rec.items()}
        x = torch.cat([s.cuda()[0] + step, s.cuda()[0] - step]).unsqueeze(1)
        loss = v.distill_loss(x, wide)["loss"][:, 0]
        num = (loss[:V] - loss[V:]) / (2 * h)
    assert (num - grad).abs().max() < 1.2e-3


@pytest.mark.parametrize("V", [3001, 100003])
def test_large_offsets(gpu, V):
    """Rows past 2^31 elements of the first."""
    K = 8
    t, s = _rows(37, 3, 1, V, "bf16")
    rec = _record(t, K, 1.0)
    dev = {k: x.cuda() for k, x in rec.items()}
    buf = torch.zeros((1 << 31) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (3, 1, V), (1 << 30, V, 1), 4097)
    x.copy_(s)
    with sv.Verifier(1, 0, V) as v:
        want = v.distill_loss_grad(s.cuda(), dev)
        a = v.distill_loss(x, dev)
        _check(s, rec, None, 1.0, "bucket", a, None)
        got = v.distill_loss_grad(x, dev, grad=x)
        assert torch.equal(x, want["grad"]) and torch.equal(got["loss"], want["loss"])


@pytest.mark.parametrize("B,n,V", [(30, 40, 2003), (30, 14, 40001), (12, 5, 100003)])
def test_many_rows_repeat_bit_for_bit(gpu, B, n, V):
    K = 16
    g = torch.Generator(device="cuda").manual_seed(5)
    x = (torch.randn(B, n, V, generator=g, device="cuda") * 3).to(torch.bfloat16)
    with sv.Verifier(1, 0, V) as v:
        rec = v.top_logits(x + torch.randn(B, n, V, generator=g, device="cuda").to(torch.bfloat16), K)
        rec["tokens"][:, ::2, 5] = rec["tokens"][:, ::2, 0]                # a token twice in every other row
        a, b = v.distill_loss_grad(x, rec), v.distill_loss_grad(x, rec)
        for k in a:
            assert torch.equal(a[k], b[k])
        cut = {k: y[7:9].contiguous() for k, y in rec.items()}
        row = v.distill_loss_grad(x[7:9], cut)
        assert torch.equal(row["grad"], a["grad"][7:9]) and torch.equal(row["loss"], a["loss"][7:9])
        cpu = {k: y[7:9].cpu() for k, y in rec.items()}
        _check(x[7:9].cpu(), cpu, None, 1.0, "bucket", {"loss": row["loss"], "flags": row["flags"]}, row["grad"])


def test_parts_and_whole_rows_agree(gpu):
    """With and without a workspace: sums in another order, so within twice
    the bounds above; here simply 2e-5 of the loss and of the largest gradient
    (two float32 log-sum-exps of 50000 terms, 250 * 2^-24 each)."""
    t, s = _rows(41, 3, 5, 50000, "f32")
    rec = {k: x.cuda() for k, x in _record(t, 32, 1.3).items()}
    with sv.Verifier(1, 0, 50000) as v:
        a = v.distill_loss_grad(s.cuda(), rec, temperature=1.3)
        l1 = v.distill_loss(s.cuda(), rec, temperature=1.3)
        _no_workspace(v)
        b = v.distill_loss_grad(s.cuda(), rec, temperature=1.3)
        l2 = v.distill_loss(s.cuda(), rec, temperature=1.3)
    for x in (l1["loss"], l2["loss"], b["loss"]):
        assert ((a["loss"] - x).abs() <= 2e-5 * x.abs() + 2e-5).all()
    assert ((a["loss"] - b["loss"]).abs() <= 2e-5 * b["loss"].abs() + 2e-5).all()
    assert (a["grad"] - b["grad"]).abs().max() <= 2e-5 * b["grad"].abs().max()
    assert (l1["lse"] - l2["lse"]).abs().max() <= 2e-5


def test_binding_refusals(gpu):
    x = torch.randn(2, 3, 64, device="cuda")
    with sv.Verifier(1, 0, 64) as v:
        rec = v.top_logits(x, 4)
        lse = v.distill_loss(x, rec)["lse"]
        cases = [lambda: v.distill_loss(x, rec, tail="none"), lambda: v.distill_loss(x, rec, temperature=0.0),
                 lambda: v.distill_loss(x, rec, weights=torch.ones(2, 2, device="cuda")),
                 lambda: v.distill_loss(x, rec, weights=torch.ones(2, 3)),
                 lambda: v.distill_loss(x[:1], rec), lambda: v.distill_loss(x.double(), rec),
                 lambda: v.distill_loss(x, {**rec, "tokens": rec["tokens"].long()}),
                 lambda: v.distill_loss(x, {**rec, "logits": rec["logits"][:, :2]}),
                 lambda: v.distill_loss(x, {"tokens": rec["tokens"], "logits": rec["logits"]}),
                 lambda: v.distill_grad(x, rec, lse[:, :2]), lambda: v.distill_grad(x, rec, lse, grad=x.bfloat16()),
                 lambda: v.distill_loss_grad(x.expand(2, 3, 64)[:, :1].expand(2, 3, 64), rec, grad=x[:, :1].expand(2, 3, 64)),
                 lambda: v.distill_loss_grad(x, rec, grad=x[:, :, :63])]
        for call in cases:
            with pytest.raises(sv.SpecvError):
                call()
        v.distill_loss(x, {"tokens": rec["tokens"], "logits": rec["logits"]}, tail="renorm")
        assert v.distill_loss(x[:0], {k: y[:0] for k, y in rec.items()})["loss"].shape == (0, 3)
