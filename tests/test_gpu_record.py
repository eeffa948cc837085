"""specv_top_logits against the float64 oracle: tokens and logits equal, ties
to the lowest token, log-sum-exps within

    (V / 256 + 40 + 6 (1 + |lse| + |max| / T)) * 2^-24

absolute: every exponential of the sum is off by less than 4 * 2^-24 relative
(its own last place and two roundings of an argument d, d e^-d < 1/2), a sum of
V positive terms in strands of at least 256 threads and a tree by
(V / 256 + 32) * 2^-24, and the joins and the logarithm by the rest.
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


def _compare(rec, z, K, T):
    """rec of one call on rows z [R, V] (CPU tensor)."""
    tok = rec["tokens"].cpu().numpy().reshape(-1, K)
    val = rec["logits"].cpu().numpy().reshape(-1, K)
    lse = rec["lse"].cpu().numpy().reshape(-1, 2)
    zz = z.double().numpy().reshape(len(tok), -1)
    V = zz.shape[1]
    for r in range(len(tok)):
        t, x, a, o = ol.top_logits(zz[r], K, T)
        assert np.array_equal(tok[r], t), r
        assert np.array_equal(val[r], x), r
        for got, want in ((lse[r, 0], a), (lse[r, 1], o)):
            if not np.isfinite(want):
                assert np.array_equal(got, want, equal_nan=True), r
                continue
            tol = (V / 256 + 40 + 6 * (1 + abs(want) + abs(zz[r][np.isfinite(zz[r])]).max() / T)) * 2.0 ** -24
            assert abs(got - want) <= tol, (r, got, want, tol)


def _run(z, K, T=1.0):
    with sv.Verifier(1, 0, z.shape[2]) as v:
        rec = v.top_logits(z.cuda(), K, T)
        torch.cuda.synchronize()
    _compare(rec, z, K, T)
    return rec


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,n,V,K,T", [
    (1, 1, 1, 1, 1.0), (1, 2, 1, 4, 1.0), (2, 3, 7, 3, 0.5), (3, 1, 64, 64, 2.0), (2, 1, 64, 100, 1.0),
    (1, 2, 255, 255, 1.0), (1, 2, 257, 256, 1.0), (2, 2, 1023, 16, 1.0), (2, 1, 4097, 1, 1.0),
    (1, 2, 8191, 256, 0.25), (2, 2, 20001, 64, 1.0), (1, 3, 50257, 50, 4.0), (2, 1, 128256, 200, 1.0),
    (1, 1, 152064, 64, 1.0), (1, 1, 200001, 7, 1.0), (1, 1, 524288, 256, 1.0)])
def test_normal_rows(gpu, dtype, B, n, V, K, T):
    rng = np.random.default_rng(V + K)
    z = torch.from_numpy(rng.normal(0, 3, (B, n, V)).astype(np.float32)).to(DTYPES[dtype])
    _run(z, K, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [63, 64, 511, 512, 513, 4095, 4096, 4104, 8192, 8193, 16383, 16384, 16385, 65536, 65537,
                               131071, 131072, 131073, 262144, 262145])
def test_sizes_at_the_edges(gpu, dtype, V):
    """Lengths where groups, steps and blocks end; the largest at both ends."""
    rng = np.random.default_rng(V)
    z = rng.normal(0, 3, (1, 2, V)).astype(np.float32)
    z[0, 1, 0] = z[0, 1, V - 1] = 30.0
    z = torch.from_numpy(z).to(DTYPES[dtype])
    for K in (2, 40):
        _run(z, K)


def _pattern(name, V, rng):
    z = rng.normal(0, 2, V).astype(np.float32)
    if name == "constant":
        z[:] = 1.25
    elif name == "two_values":
        z = np.where(rng.random(V) < 0.5, 1.0, 1.0 + 2.0 ** -6).astype(np.float32)
    elif name == "ascending":
        z = np.linspace(-4, 4, V).astype(np.float32)
    elif name == "descending":
        z = np.linspace(4, -4, V).astype(np.float32)
    elif name == "block":                    # the largest all in one run of neighbours
        z[V // 3:V // 3 + 400] += 20
    elif name == "stride":                   # and all in one residue class
        z[5::1024] += 20
        z[5::8192] += 5
    elif name == "zeros":
        z = np.where(rng.random(V) < 0.5, 0.0, -0.0).astype(np.float32)
    elif name == "masked":                   # a grammar that leaves few tokens
        keep = rng.integers(0, V, 9)
        m = np.full(V, -np.inf, np.float32)
        m[keep] = z[keep]
        z = m
    elif name == "one":
        z[:] = -np.inf
        z[V // 2] = -7.0
    elif name == "lowest":                   # masks of the type's lowest value
        z[rng.random(V) < 0.999] = -3.3895313892515355e38
    elif name == "peaked":                   # a rest far below the record
        z[:] = -200.0 + z
        z[:3] = 50.0
    elif name == "negative":
        z = -np.abs(z) - 50
    return z


PATTERNS = ["constant", "two_values", "ascending", "descending", "block", "stride", "zeros", "masked", "one",
            "lowest", "peaked", "negative"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [700, 9001, 131072, 200000])
def test_patterned_rows(gpu, dtype, V):
    rng = np.random.default_rng(V)
    z = torch.from_numpy(np.stack([_pattern(p, V, rng) for p in PATTERNS])[:, None]).to(DTYPES[dtype])
    for K in (1, 3, 64, 256):
        print(V, K, flush=True)
        _run(z, K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3, 5000, 140000])
def test_rows_without_a_record(gpu, dtype, V):
    z = torch.zeros(5, 1, V, dtype=DTYPES[dtype])
    z[0, 0, V - 1] = float("nan")
    z[1, 0, 0] = float("inf")
    z[2] = -float("inf")
    z[3, 0, V // 2] = -float("nan")
    _run(z, 4)


@pytest.mark.parametrize("V", [1000, 30001])
def test_strides_and_broadcast(gpu, V):
    g = torch.Generator().manual_seed(V)
    z = torch.randn(3, 2, V, generator=g).to(torch.bfloat16)
    with sv.Verifier(1, 0, V) as v:
        want = v.top_logits(z.cuda(), 40)
        _compare(want, z, 40, 1.0)
        buf = torch.full((6 * (V + 7) + 5,), float("nan"), dtype=torch.bfloat16, device="cuda")
        for strides, off in (((2 * (V + 7), V + 7, 1), 1), ((V + 1, 3 * (V + 1), 1), 3)):
            x = torch.as_strided(buf, (3, 2, V), strides, off)
            x.copy_(z)
            got = v.top_logits(x, 40)
            assert torch.equal(got["tokens"], want["tokens"]) and torch.equal(got["logits"], want["logits"])
            _compare(got, z, 40, 1.0)
            buf.fill_(float("nan"))
        one = v.top_logits(z[:1, :1].cuda().expand(3, 2, V), 40)
        assert torch.equal(one["tokens"], want["tokens"][:1, :1].expand(3, 2, 40))


def test_large_offsets(gpu):
    """Rows past 2^31 elements of the first."""
    V = 30001
    g = torch.Generator().manual_seed(4)
    z = (torch.randn(3, 1, V, generator=g) * 3).to(torch.bfloat16)
    buf = torch.zeros((1 << 31) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (3, 1, V), (1 << 30, V, 1), 4097)
    x.copy_(z)
    with sv.Verifier(1, 0, V) as v:
        _compare(v.top_logits(x, 50), z, 50, 1.0)


def test_many_rows_repeat_bit_for_bit(gpu):
    g = torch.Generator(device="cuda").manual_seed(1)
    z = (torch.randn(40, 25, 5003, generator=g, device="cuda") * 3).to(torch.bfloat16)
    with sv.Verifier(1, 0, 5003) as v:
        a, b = v.top_logits(z, 33, 0.9), v.top_logits(z, 33, 0.9)
        for k in a:
            assert torch.equal(a[k], b[k])
        _compare({k: x[:3] for k, x in a.items()}, z[:3].cpu(), 33, 0.9)
        row = v.top_logits(z[17:18, 4:5], 33, 0.9)                        # a row does not depend on its neighbours
        assert torch.equal(row["tokens"][0, 0], a["tokens"][17, 4])


def test_binding_refusals(gpu):
    x = torch.zeros(2, 3, 64, device="cuda")
    with sv.Verifier(1, 0, 64) as v:
        for call in (lambda: v.top_logits(x, 0), lambda: v.top_logits(x, 257), lambda: v.top_logits(x, 4, 0.0),
                     lambda: v.top_logits(x.half(), 4), lambda: v.top_logits(x[0], 4),
                     lambda: v.top_logits(torch.zeros(1, 1, 65, device="cuda"), 4)):
            with pytest.raises(sv.SpecvError):
                call()
        assert v.top_logits(x[:0], 4)["tokens"].shape == (0, 3, 4)
