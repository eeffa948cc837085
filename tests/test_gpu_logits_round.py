"""The logits operators used together, as a server that trains its drafter
uses them: adjusted rows, verify, history, record, loss and gradient; captured
into a graph and replayed; on a stream of their own; next to verify calls."""

import numpy as np
import pytest
import torch

import oracle
from oracle import logits as ol
import synth
import speculative_decoding_verification_sampling_amd as sv
from parity import compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    sv.load_library()
    return torch.device("cuda:0")


def test_rounds_with_penalties_masks_and_a_training_step(gpu):
    """Three rounds: drafts drawn one position at a time from adjusted draft
    rows, verified against adjusted target rows, emitted tokens taken into the
    histories, and the drafter's gradient against the record of the raw target
    rows.  Every piece is compared with the oracle of its own inputs."""
    B, gamma, V, K = 4, 3, 3001, 16
    rng = np.random.default_rng(2)
    rep, pres, freq = np.float32(1.3), np.float32(0.4), np.float32(0.2)
    pen = sv.make_penalties(B, rep, pres, freq, [5, 0, 3, 1])
    slots = torch.tensor([5, 0, 3, 1], dtype=torch.int32, device="cuda")
    h = sv.TokenHistory(6, V)
    T = np.array([1.0, 0.7, 0.0, 1.0], np.float32)
    rp = sv.make_row_params(B, T)
    prompt = rng.integers(0, V, (B, 30)).astype(np.int32)
    past = [{} for _ in range(B)]
    with sv.Verifier(B, gamma, V) as v:
        v.history_reset(h, slots)
        v.history_add(h, slots, torch.from_numpy(prompt).cuda(), prompt=True)
        for step in range(3):
            t, d = synth.make_logits(rng, B, gamma, V, 3.0, 1.0, boost_count=20)
            target, draft = torch.from_numpy(t).cuda(), torch.from_numpy(d).cuda()
            allowed = rng.random((B, gamma + 1, V)) < 0.8
            mask = sv.pack_token_mask(torch.from_numpy(allowed).cuda())
            tokens = torch.zeros(B, gamma, dtype=torch.int32, device="cuda")
            drawn = {"tokens": tokens, "stats": torch.zeros(B, gamma, 4, device="cuda")}
            adj_draft = torch.empty_like(draft)
            for i in range(gamma):                   # the drafter sees the drafts before its position
                v.adjust_logits(draft[:, i:i + 1], pen, h, tokens, i, mask=mask[:, i:i + 1],
                                out=adj_draft[:, i:i + 1])
                v.sample_draft(adj_draft[:, i:i + 1], rp, 100 + step, step, pos0=i, out=drawn)
            adj = v.adjust_logits(target, pen, h, tokens, mask=mask)
            rec = v.top_logits(target, K)
            out = v.verify_sample_qstats(adj, adj_draft, drawn["stats"], tokens, rp, 7, step)
            both = v.distill_loss_grad(draft, rec, tail="bucket")
            v.history_add(h, slots, out["out_tokens"], out["num_emitted"])
            torch.cuda.synchronize()
            toks = tokens.cpu().numpy()
            for b in range(B):
                for i in range(gamma + 1):
                    for got, z in ((adj, t), (adj_draft, d)):
                        if i >= got.shape[1]:
                            continue
                        want = ol.adjust_row(z[b, i], past[b], prompt[b].tolist(), toks[b, :i].tolist(), float(rep),
                                             float(pres), float(freq), (), allowed[b, i])
                        g = got[b, i].double().cpu().numpy()
                        assert np.array_equal(np.isfinite(g), np.isfinite(want))
                        f = np.isfinite(want)
                        assert np.abs(g[f] - want[f]).max() < 6 * 2.0 ** -24 * 64
                for i in range(gamma):
                    r = {k: x[b, i].cpu().numpy() for k, x in rec.items()}
                    loss, grad, _, _ = ol.distill(d[b, i], r["tokens"], r["logits"].astype(float),
                                                  r["lse"].astype(float), 1.0, "bucket")
                    assert abs(both["loss"][b, i].item() - loss) < 1e-4
                    assert np.abs(both["grad"][b, i].double().cpu().numpy() - grad).max() < 1e-5
            orc = oracle.verify_sample(adj.cpu().numpy(), adj_draft.cpu().numpy(), toks, T, 0, 1.0,
                                       np.zeros(B, np.int32), 7, step)
            compare(out, orc, toks, adj.cpu().numpy(), adj_draft.cpu().numpy(),
                    {"temperature": T, "top_k": np.zeros(B, np.int32), "top_p": np.ones(B, np.float32)}).assert_ok(0.3)
            emitted, num = out["out_tokens"].cpu().numpy(), out["num_emitted"].cpu().numpy()
            for b in range(B):
                for x in emitted[b, :num[b]]:
                    past[b][int(x)] = past[b].get(int(x), 0) + 1
                assert int(h.counts[[5, 0, 3, 1][b]].sum()) == sum(past[b].values())


@pytest.mark.parametrize("V", [20001, 100003])          # whole rows; parts of rows, with a workspace
def test_captured_and_replayed(gpu, V):
    """All operators in one graph, replayed on new contents with eager work
    and synchronizations between, each replay equal to eager calls."""
    B, gamma, K = 6, 3, 32
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    target = (3 * rnd(B, gamma + 1, V)).to(torch.bfloat16)
    draft = (3 * rnd(B, gamma, V)).to(torch.bfloat16)
    tokens = torch.randint(0, V, (B, gamma), generator=g, device="cuda", dtype=torch.int32)
    words = (V + 31) // 32
    mask = torch.randint(-(1 << 31), (1 << 31) - 1, (B, gamma + 1, words), generator=g, device="cuda",
                         dtype=torch.int64).to(torch.int32)
    bias = sv.make_bias([[(7, 1.0), (V - 1, -2.0), (7, 0.5)]] * B)
    pen = sv.make_penalties(B, 1.2, 0.3, 0.1)
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    weights = torch.rand(B, gamma, generator=g, device="cuda")
    rp = sv.make_row_params(B, 0.9)
    v = sv.Verifier(B, gamma, V)
    v.set_profiling(True)                                        # events are left out under capture

    def body(h, adj, grad):
        v.adjust_logits(target, pen, h, tokens, bias=bias, mask=mask, out=adj)
        rec = v.top_logits(target, K, 1.5)
        loss = v.distill_loss(draft, rec, weights, 1.5, "renorm")
        g1 = v.distill_grad(draft, rec, loss["lse"], weights, 1.5, "renorm")
        both = v.distill_loss_grad(draft, rec, weights, 1.5, "bucket", grad=grad)
        out = v.verify_point_mass(adj, tokens, rp, 3)
        v.history_reset(h, slots[:2])
        v.history_add(h, slots, out["out_tokens"])
        return [adj, rec["tokens"], rec["logits"], rec["lse"], loss["loss"], loss["lse"], g1, both["loss"],
                both["grad"], out["out_tokens"], h.counts, h.seen]

    hist = sv.TokenHistory(B, V)
    adj, grad = torch.empty_like(target), torch.empty_like(draft)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        body(sv.TokenHistory(B, V), adj, grad)                   # warm-up on other histories
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = body(hist, adj, grad)
    eager_hist = sv.TokenHistory(B, V)
    hist.counts.zero_()
    hist.seen.zero_()
    for r in range(4):
        target.copy_((3 * rnd(B, gamma + 1, V)).to(torch.bfloat16))
        draft.copy_((2 * rnd(B, gamma, V)).to(torch.bfloat16))
        tokens.copy_(torch.randint(0, V, (B, gamma), generator=g, device="cuda", dtype=torch.int32))
        graph.replay()
        got = [x.clone() for x in outs]
        torch.cuda.synchronize()
        want = body(eager_hist, torch.empty_like(adj), torch.empty_like(grad))
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (r, k)
    v.close()


@pytest.mark.parametrize("B,V", [(16, 50000), (8, 100003)])
def test_two_streams_at_once(gpu, B, V):
    """Calls of one handle on two streams, next to each other and to a verify
    call, give what they give alone."""
    gamma, K = 4, 64
    g = torch.Generator(device="cuda").manual_seed(12)
    xs = [(3 * torch.randn(B, gamma + 1, V, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    tok = torch.randint(0, V, (B, gamma), generator=g, device="cuda", dtype=torch.int32)
    rp = sv.make_row_params(B, 1.0)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def body(v, x):
        rec = v.top_logits(x, K)
        o = v.distill_loss_grad(x, rec)
        a = v.adjust_logits(x, sv_pen, None, tok)
        return [rec["tokens"], rec["lse"], o["loss"], o["grad"], a]

    sv_pen = sv.make_penalties(B, 1.5, 0.5, 0.5)
    with sv.Verifier(B, gamma, V) as v:
        want = [[t.clone() for t in body(v, x)] for x in xs]
        ref = v.verify_point_mass(xs[0], tok, rp, 5)["out_tokens"].clone()
        torch.cuda.synchronize()
        for _ in range(3):
            got = []
            for s, x in zip(streams, xs):
                with torch.cuda.stream(s):
                    got.append(body(v, x))
            out = v.verify_point_mass(xs[0], tok, rp, 5)["out_tokens"]
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
            for a, b in zip(got, want):
                for p, q in zip(a, b):
                    assert torch.equal(p, q)


def test_profiling_counts_the_calls(gpu):
    x = torch.randn(2, 2, 5000, device="cuda")
    with sv.Verifier(2, 2, 5000) as v:
        v.set_profiling(True)
        rec = v.top_logits(x, 8)
        v.distill_loss(x, rec)
        v.adjust_logits(x, sv.make_penalties(2))
        n, ms = v.profile()
        assert n == 3 and ms > 0


@pytest.mark.parametrize("tail", ["bucket", "renorm"])
def test_training_step_of_a_linear_drafter(gpu, tail):
    """The gradient taken on into a model's weights by backward, against the
    float64 gradient of the same loss by torch on the CPU.  The logits'
    gradients are off by at most 4e-6 of their largest (float32 sums of 2000
    terms and a few roundings), a sum of 12 rows of them against |x| < 4 by
    no more relative to the sum of magnitudes."""
    B, n, D, V, K, T = 3, 4, 16, 2000, 12, 1.5
    g = torch.Generator().manual_seed(3)
    x, W = torch.randn(B, n, D, generator=g), torch.randn(V, D, generator=g) * 0.5
    teacher = torch.randn(B, n, V, generator=g) * 3
    w = torch.rand(B, n, generator=g)
    w[1, 2] = 0.0
    with sv.Verifier(1, 0, V) as v:
        rec = v.top_logits(teacher.cuda(), K, T)
        Wd = W.cuda().requires_grad_()
        logits = x.cuda() @ Wd.t()
        out = v.distill_loss_grad(logits, rec, weights=w.cuda(), temperature=T, tail=tail)
        logits.backward(out["grad"])
    W64 = W.double().requires_grad_()
    logq = torch.log_softmax(x.double() @ W64.t() / T, -1)
    t = teacher.double() / T
    idx = rec["tokens"].cpu().long()
    logp = t.gather(-1, idx) - torch.logsumexp(t if tail == "bucket" else t.gather(-1, idx), -1, keepdim=True)
    loss = (logp.exp() * (logp - logq.gather(-1, idx))).sum(-1)
    if tail == "bucket":
        po = 1 - logp.exp().sum(-1)
        qo = 1 - logq.exp().gather(-1, idx).sum(-1)
        loss = loss + po * (po.log() - qo.log())
    (loss * w.double()).sum().backward()
    assert (out["loss"].cpu().double() - loss.detach() * w).abs().max() < 2e-5
    scale = (w.double().sum() / T) * 4
    assert (Wd.grad.cpu().double() - W64.grad).abs().max() < 4e-6 * scale
