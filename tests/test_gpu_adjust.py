"""specv_adjust_logits and the token histories against the float64 oracle.

Tolerance: the steps are float32 operations rounded to nearest, so an adjusted
logit is off by at most 2^-24 of each intermediate value (five of them, none
above A = |z| r + |z / r| + f c + |a| + sum |bias|, with one more per bias
entry of the token), and by half a step of the output type at the end.  Logits
that no step names must keep their bits.
"""

import numpy as np
import pytest
import torch

from oracle import logits as ol
import speculative_decoding_verification_sampling_amd as sv

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    sv.load_library()
    return torch.device("cuda:0")


def _dicts(counts, seen, V, slot):
    """counts {token: n} and the seen tokens of one slot, from the tensors."""
    if slot < 0 or slot >= counts.shape[0]:
        return {}, []
    c = counts[slot].cpu().numpy()
    bits = np.unpackbits(seen[slot].cpu().numpy().view(np.uint8), bitorder="little")[:V]
    used = np.nonzero(bits)[0]
    return {int(t): int(c[t]) for t in used if c[t]}, used.tolist()


def _check(got, z, dtype, V, B, n, pos0, prm, counts, seen, drafts, bias, allowed):
    """Compare with the oracle, row by row."""
    u = torch.finfo(DTYPES[dtype]).eps / 2
    rep, pres, freq, slot = prm
    for b in range(B):
        c, used = _dicts(counts, seen, V, slot[b]) if counts is not None else ({}, [])
        for i in range(n):
            before = drafts[b, :pos0 + i].tolist() if drafts is not None else []
            zz = z[b, i].double().numpy()
            on = prm is not None and counts is not None or drafts is not None
            want = ol.adjust_row(zz, c, used, before, rep[b] if on else 1.0, pres[b], freq[b],
                                 bias[b] if bias else (), None if allowed is None else allowed[b, i].numpy())
            g = got[b, i].double().cpu().numpy()
            touched = set(used) | {t for t in before if 0 <= t < V} | {t for t, _ in (bias[b] if bias else ())
                                                                      if 0 <= t < V}
            idx = np.array(sorted(touched), dtype=int)
            same = np.ones(V, bool)
            same[idx] = False
            if allowed is not None:
                same &= allowed[b, i].numpy()
                assert (g[~allowed[b, i].numpy()] == -np.inf).all()
            assert np.array_equal(g[same], zz[same], equal_nan=True)
            if allowed is not None:
                idx = idx[allowed[b, i].numpy()[idx]]
            if len(idx) == 0:
                continue
            n_bias = len(bias[b]) if bias else 0
            n_use = max([c.get(t, 0) for t in c] + [0]) + len(before)
            A = np.abs(zz[idx]) * max(rep[b], 1 / rep[b]) + abs(freq[b]) * n_use + abs(pres[b])
            if bias:
                A = A + sum(abs(x) for _, x in bias[b])
            tol = u * np.abs(want[idx]) + (5 + n_bias) * 2.0 ** -24 * A + 1e-38
            fin = np.isfinite(want[idx])
            assert np.array_equal(g[idx][~fin], want[idx][~fin], equal_nan=True)
            assert (np.abs(g[idx] - want[idx])[fin] <= tol[fin]).all(), (b, i)


def _setup(seed, B, n, V, dtype, pos0=0, S=None, used=20):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)).to(DTYPES[dtype])
    S = B + 2 if S is None else S
    h = sv.TokenHistory(S, V)
    tok = torch.from_numpy(rng.integers(0, V, (S, used)).astype(np.int32)).cuda()
    with sv.Verifier(1, 0, V) as v:
        slots = torch.arange(S, dtype=torch.int32, device="cuda")
        v.history_add(h, slots, tok[:, :used // 2].contiguous(), prompt=True)
        v.history_add(h, slots, tok[:, used // 2:])
    rep = rng.uniform(0.7, 1.8, B).astype(np.float32)
    pres, freq = rng.normal(0, 1, (2, B)).astype(np.float32)
    slot = rng.permutation(S)[:B].astype(np.int32)
    drafts = rng.integers(0, V, (B, max(pos0 + n - 1, 1))).astype(np.int32)
    if drafts.shape[1] > 2:
        drafts[:, 2] = drafts[:, 0]                                    # the same draft twice
    drafts[0, 0] = V + 3                                               # outside the vocabulary
    bias = [[(int(t), float(x)) for t, x in zip(rng.integers(0, V, k), rng.normal(0, 2, k).astype(np.float32))]
            for k in rng.integers(0, 6, B)]
    bias[-1] = [(int(drafts[-1, 0]), 1.0), (V - 1, -2.0), (V - 1, 0.5), (V, 3.0), (-1, 3.0)]
    allowed = torch.from_numpy(rng.random((B, n, V)) < 0.7)
    allowed[0, 0] = False                                              # a row the mask leaves empty
    if B > 1:
        allowed[1] = True
    return z, h, (rep, pres, freq, slot), drafts, bias, allowed


SHAPES = [(1, 2, 2048, 0), (2, 3, 2056, 0), (1, 5, 4096, 3), (1, 32, 65, 31), (300, 2, 2050, 0), (1, 1, 1, 0), (2, 3, 7, 0), (3, 2, 8, 1), (2, 4, 33, 2), (2, 6, 2047, 0), (3, 1, 2049, 4), (2, 3, 5001, 0),
          (2, 32, 129, 0), (2, 2, 131, 30)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,n,V,pos0", SHAPES)
def test_everything_at_once(gpu, dtype, B, n, V, pos0):
    z, h, prm, drafts, bias, allowed = _setup(7, B, n, V, dtype, pos0)
    with sv.Verifier(1, 0, V) as v:
        args = dict(penalties=sv.make_penalties(B, *prm), history=h, draft_tokens=torch.from_numpy(drafts).cuda(),
                    pos0=pos0, bias=sv.make_bias(bias), mask=sv.pack_token_mask(allowed.cuda()))
        x = z.cuda()
        got = v.adjust_logits(x, **args)
        assert torch.equal(x.cpu(), z)                                 # the input stays
        v.adjust_logits(x, out=x, **args)
        assert torch.equal(x.view(torch.uint8), got.view(torch.uint8))  # in place: the same bits
    _check(got, z, dtype, V, B, n, pos0, prm, h.counts, h.seen, drafts, bias, allowed)


@pytest.mark.parametrize("parts", ["penalties", "drafts", "bias", "mask", "none"])
def test_each_part_alone(gpu, parts):
    B, n, V, dtype = 3, 4, 3001, "bf16"
    z, h, prm, drafts, bias, allowed = _setup(11, B, n, V, dtype)
    off = (np.ones(B, np.float32), np.zeros(B, np.float32), np.zeros(B, np.float32), prm[3])
    kw, chk = {}, dict(prm=off, counts=None, seen=None, drafts=None, bias=None, allowed=None)
    if parts == "penalties":
        kw = dict(penalties=sv.make_penalties(B, *prm), history=h)
        chk.update(prm=prm, counts=h.counts, seen=h.seen)
    elif parts == "drafts":
        kw = dict(penalties=sv.make_penalties(B, *prm), draft_tokens=torch.from_numpy(drafts).cuda())
        chk.update(prm=prm, drafts=drafts)
    elif parts == "bias":
        kw = dict(bias=sv.make_bias(bias))
        chk.update(bias=bias)
    elif parts == "mask":
        kw = dict(mask=sv.pack_token_mask(allowed.cuda()))
        chk.update(allowed=allowed)
    with sv.Verifier(1, 0, V) as v:
        got = v.adjust_logits(z.cuda(), **kw)
    _check(got, z, dtype, V, B, n, 0, chk["prm"], chk["counts"], chk["seen"], chk["drafts"], chk["bias"],
           chk["allowed"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_special_values(gpu, dtype):
    V, B, n = 40, 1, 2
    z = torch.zeros(B, n, V, dtype=DTYPES[dtype])
    z[0, 0, :8] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, torch.finfo(DTYPES[dtype]).min,
                                torch.finfo(DTYPES[dtype]).max, 1e-30, -1e-30])
    z[0, 1] = z[0, 0]
    h = sv.TokenHistory(1, V)
    allowed = torch.ones(B, n, V, dtype=torch.bool)
    allowed[0, 1, :4] = False
    with sv.Verifier(1, 0, V) as v:
        slots = torch.zeros(1, dtype=torch.int32, device="cuda")
        v.history_add(h, slots, torch.tensor([[2, 3, 4, 5, 6, 7]], dtype=torch.int32, device="cuda"))
        got = v.adjust_logits(z.cuda(), penalties=sv.make_penalties(1, 2.0, 0.0, 0.0), history=h,
                              mask=sv.pack_token_mask(allowed.cuda())).cpu()
    assert torch.isnan(got[0, 0, 0]) and got[0, 0, 1] == float("inf") and got[0, 0, 2] == -float("inf")
    assert got[0, 0, 3] == 0 and got[0, 0, 4] == -float("inf")         # lowest value times two
    assert got[0, 0, 5] == torch.finfo(DTYPES[dtype]).max / 2
    assert (got[0, 1, :4] == -float("inf")).all()                      # NaN and +inf masked
    assert torch.equal(got[0, 1, 4:], got[0, 0, 4:])


def test_strides_broadcasts_and_slots(gpu):
    """Odd row starts, padded rows, position-major rows, broadcast logits and
    masks, slots shared, negative and beyond the histories."""
    B, n, V = 4, 3, 1001
    z, h, prm, drafts, bias, allowed = _setup(13, B, n, V, "bf16", S=5)
    prm = (*prm[:3], np.array([2, 2, -1, 5], np.int32))
    kw = dict(penalties=sv.make_penalties(B, *prm), history=h, draft_tokens=torch.from_numpy(drafts).cuda(),
              bias=sv.make_bias(bias))
    full_mask = sv.pack_token_mask(allowed.cuda())
    with sv.Verifier(1, 0, V) as v:
        want = v.adjust_logits(z.cuda(), mask=full_mask, **kw)
        _check(want, z, "bf16", V, B, n, 0, prm, h.counts, h.seen, drafts, bias, allowed)
        wide = torch.zeros(B * n * 1024 + 8, dtype=torch.bfloat16, device="cuda")
        for shape, strides, off in (((B, n, V), (n * 1024, 1024, 1), 1), ((B, n, V), (1003, 4 * 1003, 1), 3)):
            x = torch.as_strided(wide, shape, strides, off)
            x.copy_(z)
            keep = wide.clone()
            got = v.adjust_logits(x, mask=full_mask, **kw)
            assert torch.equal(got, want)
            v.adjust_logits(x, mask=full_mask, out=x, **kw)
            assert torch.equal(x, want)
            outside = torch.ones_like(wide, dtype=torch.bool)
            torch.as_strided(outside, shape, strides, off).fill_(False)
            assert torch.equal(wide[outside], keep[outside])           # nothing behind the rows is written
        W = full_mask.shape[2]
        padded = torch.full((n, B, W + 5), -1, dtype=torch.int32, device="cuda")     # mask rows apart, other order
        padded[:, :, 2:2 + W] = full_mask.transpose(0, 1)
        got = v.adjust_logits(z.cuda(), mask=padded.transpose(0, 1)[:, :, 2:2 + W], **kw)
        assert torch.equal(got, want)
        one = z[:1, :1].cuda().expand(B, n, V)                         # broadcast logits and mask
        m1 = full_mask[1:2, :1].expand(B, n, -1)
        got = v.adjust_logits(one, mask=m1, **kw)
        assert torch.equal(got, v.adjust_logits(one.contiguous(), mask=m1.contiguous(), **kw))


def test_many_biases_on_one_row(gpu):
    """More entries than a workgroup takes at once, many for the same tokens."""
    V, rng = 4099, np.random.default_rng(3)
    z = torch.from_numpy(rng.normal(0, 1, (2, 2, V)).astype(np.float32))
    bias = [[(int(t), float(x)) for t, x in zip(rng.integers(0, k, 1500), rng.normal(0, 1, 1500).astype(np.float32))]
            for k in (V, 40)]
    off = (np.ones(2, np.float32), np.zeros(2, np.float32), np.zeros(2, np.float32), np.zeros(2, np.int32))
    with sv.Verifier(1, 0, V) as v:
        got = v.adjust_logits(z.cuda(), bias=sv.make_bias(bias))
        again = v.adjust_logits(z.cuda(), bias=sv.make_bias(bias))
        # offsets that point outside the entries are cut
        o, t, x = sv.make_bias(bias)
        bad = o.clone()
        bad[0], bad[2] = -5, 1 << 30
        assert torch.equal(v.adjust_logits(z.cuda(), bias=(bad, t, x)), got)
    assert torch.equal(got, again)
    _check(got, z, "f32", V, 2, 2, 0, off, None, None, None, bias, None)


def test_large_offsets(gpu):
    """Rows whose elements lie past 2^31 of the first, and a history past 2^31 counts."""
    V, rows = 4000, 3
    buf = torch.zeros((1 << 31) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (rows, 1, V), (1 << 30, V, 1), 4096)
    x.copy_(torch.randn(rows, 1, V, device="cuda"))
    S = (1 << 31) // V + 10
    counts = torch.zeros(S, V, dtype=torch.int32, device="cuda")
    h = sv.TokenHistory(S, V, counts=counts, seen=torch.zeros(S, V // 32, dtype=torch.int32, device="cuda"))
    slot = [S - 1, S - 2, 0]
    with sv.Verifier(1, 0, V) as v:
        v.history_add(h, torch.tensor(slot, dtype=torch.int32, device="cuda"),
                      torch.tensor([[1, 2], [3, 3], [V - 1, 5]], dtype=torch.int32, device="cuda"))
        assert counts[S - 2, 3] == 2 and counts[S - 1, 2] == 1
        got = v.adjust_logits(x, penalties=sv.make_penalties(rows, 1.0, 0.0, 1.0, slot), history=h)
        want = x.float()
        for b, t, c in ((0, 1, 1), (0, 2, 1), (1, 3, 2), (2, V - 1, 1), (2, 5, 1)):
            want[b, 0, t] -= c
        assert torch.equal(got, want.to(torch.bfloat16))
        v.adjust_logits(x, penalties=sv.make_penalties(rows, 1.0, 0.0, 1.0, slot), history=h, out=x)
        assert torch.equal(x, got)


def test_history_against_numpy(gpu):
    rng = np.random.default_rng(21)
    for B, n, V, S in ((1, 1, 1, 1), (3, 7, 31, 4), (5, 300, 1000, 3), (2, 5000, 257, 2), (3, 511, 70000, 2),
                       (3, 512, 70000, 2), (2, 40000, 300000, 2), (2, 33000, 524288, 2), (3, 16385, 3, 2)):
        h = sv.TokenHistory(S, V)
        slots = rng.integers(-1, S + 1, B).astype(np.int32)             # the same slot twice, slots outside
        tok = rng.integers(-2, V + 2, (B, n)).astype(np.int32)
        length = rng.integers(-1, n + 3, B).astype(np.int32)
        counts, seen = np.zeros((S, V), np.int32), np.zeros((S, (V + 31) // 32 * 32), np.uint8)
        with sv.Verifier(1, 0, V) as v:
            for prompt in (True, False, False):
                wide = torch.full((B, n + 3), 7, dtype=torch.int32, device="cuda")
                wide[:, :n] = torch.from_numpy(tok).cuda()
                v.history_add(h, torch.from_numpy(slots).cuda(), wide[:, :n],
                              None if prompt else torch.from_numpy(length).cuda(), prompt=prompt)
                for b, s in enumerate(slots):
                    if not 0 <= s < S:
                        continue
                    t = tok[b, :n if prompt else min(max(length[b], 0), n)]
                    t = t[(t >= 0) & (t < V)]
                    seen[s, t] = 1
                    if not prompt:
                        counts[s] += np.bincount(t, minlength=V).astype(np.int32)
            assert np.array_equal(h.counts.cpu().numpy(), counts)
            assert np.array_equal(h.seen.cpu().numpy(), np.packbits(seen, axis=1, bitorder="little").view(np.int32))
            gone = torch.tensor([0, S, 0, -3], dtype=torch.int32, device="cuda")
            v.history_reset(h, gone)
            counts[0] = 0
            seen[0] = 0
            assert np.array_equal(h.counts.cpu().numpy(), counts)
            assert np.array_equal(h.seen.cpu().numpy(), np.packbits(seen, axis=1, bitorder="little").view(np.int32))


def test_refusals_of_the_binding(gpu):
    x = torch.zeros(2, 3, 64, device="cuda")
    pen = sv.make_penalties(2)
    with sv.Verifier(1, 0, 64) as v:
        bad = [dict(out=torch.zeros(2, 3, 64)), dict(out=torch.zeros(2, 3, 63, device="cuda")),
               dict(out=torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")),
               dict(penalties=sv.make_penalties(3)), dict(penalties=pen, history=sv.TokenHistory(2, 63)),
               dict(history=sv.TokenHistory(2, 64)), dict(penalties=pen, draft_tokens=torch.zeros(2, 1, dtype=torch.int32, device="cuda")),
               dict(mask=torch.zeros(2, 3, 3, dtype=torch.int32, device="cuda")),
               dict(mask=torch.zeros(2, 3, 2, dtype=torch.int64, device="cuda")), dict(pos0=32),
               dict(bias=sv.make_bias([None])), dict(out=x.flip(0).transpose(0, 0)[:, :1].expand(2, 3, 64))]
        for kw in bad:
            with pytest.raises(sv.SpecvError):
                v.adjust_logits(x, **kw)
        with pytest.raises(sv.SpecvError):
            v.adjust_logits(torch.zeros(2, 3, 65, device="cuda"))        # V above the handle's maximum
        with pytest.raises(sv.SpecvError):
            v.adjust_logits(x.double())
        assert v.adjust_logits(x[:0]).shape == (0, 3, 64)
        assert v.adjust_logits(x[:, :0]).shape == (2, 0, 64)
