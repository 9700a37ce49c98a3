"""The token loop's operators at the borders of their definitions: exact ties of
codes, the largest weights."""
import math

import pytest

torch = pytest.importorskip("torch")
import token_plain as P  # noqa: E402

pytestmark = pytest.mark.gpu
F64 = torch.float64
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_state_space_mamba2_b200 import build, lib
    build.build()
    lib.load()
    return lib


# ------------------------------------------------------------------ norm
def row_of(first, total, top, K):
    """[K] integers that begin with `first` and top, none above top, whose squares
    sum to `total`."""
    n = [top, *first]
    left = total - sum(v * v for v in n)
    while left > 0:
        n.append(min(top, math.isqrt(left)))
        left -= n[-1] ** 2
    assert left == 0 and len(n) <= K
    return torch.tensor(n + [0] * (K - len(n)), dtype=F64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_norm_on_exact_ties(lib, kind, dtype):
    """Rows of mean square 4^j whose largest element is 448 or 127 times a power of
    two: 1 / rms and the scale are powers of two, every step is exact, and the
    arguments of the codes lie in the middle between two of them."""
    K = 128
    if kind == "e4m3":  # s = 2^-7, elements in units of 2^-18: arguments in units of 2^-11
        ties = [k * 2 ** e for k in range(17, 32, 2) for e in (3, 7, 10)]   # of normal codes
        ties += [2 * k for k in range(1, 16, 2)]                           # of subnormal ones
        n, unit = row_of(ties, K << 36, 7 << 17, K), 2.0 ** -18
    else:               # s = 2^-5, elements in units of 2^-6: arguments in halves
        n, unit = row_of([1, 3, 5, 7, 9, 61, 101, 131, 151], K << 12, 254, K), 2.0 ** -6
        ties = [1, 3, 5, 7, 9, 61, 101, 131, 151]
    x = torch.stack([n, -n, n * 8, -n / 32]) * unit
    if dtype == torch.bfloat16:  # the elements of at most 8 bits; the rest comes as the residual
        part = x.to(dtype)
        x, res = part.cuda(), (x - part.to(F64)).float().cuda()
    else:
        x, res = x.float().cuda(), None
    w = torch.ones(K, device="cuda")
    q = torch.zeros(4, K, device="cuda").to(E4M3 if kind == "e4m3" else torch.int8)
    s = torch.empty((4, 1) if kind == "e4m3" else (4,), device="cuda")
    lib.add_norm_quant(x, w, q, s, residual=res, eps=1e-30)
    lib.sync_status()
    r, codes, scales, sure = P.norm(x, res, w, 1e-30, kind)
    assert torch.equal(r.cpu().to(F64), torch.stack([n, -n, n * 8, -n / 32]) * unit)
    assert bool((scales == (2.0 ** -7 if kind == "e4m3" else 2.0 ** -5)).all())
    assert int((sure == 0).sum()) >= 4 * len(ties)
    assert torch.equal(s, scales) and torch.equal(q.float().to(F64), codes)


# ------------------------------------------------------------------ prepared weights
SCALES = [1, 3, 49, 75, 77, 91, 93, 99, 103, 147, 555, 599]


def test_prepared_weights_on_exact_ties(lib):
    """Blocks whose scale is a small integer: W / s is exactly in the middle between
    two codes, which goes to the even one."""
    W = torch.zeros(128, 128 * len(SCALES), dtype=F64)
    t = torch.tensor([k / 16 * 2.0 ** e for k in range(17, 32, 2) for e in (-6, -5, 0, 7)]
                     + [k / 1024 for k in range(1, 16, 2)], dtype=F64)
    for i, j in enumerate(SCALES):
        W[0, 128 * i] = 448 * j
        W[1, 128 * i:128 * i + len(t)] = j * t
        W[2, 128 * i:128 * i + len(t)] = -j * t
    assert torch.equal(W.float().to(F64), W)
    q, s = torch.zeros(W.shape, device="cuda").to(E4M3), torch.zeros(1, len(SCALES), device="cuda")
    lib.prepare_linear_fp8(W.float().cuda(), q, s)
    lib.sync_status()
    assert s[0].tolist() == SCALES
    want = P.e4m3_round(W / s.cpu().to(F64).repeat_interleave(128, 1))
    assert torch.equal(q.float().cpu().to(F64), want)


def test_prepared_weights_of_the_largest_magnitudes(lib):
    """Finite weights are no error however large; a NaN or an infinity is one."""
    top = torch.finfo(torch.float32).max
    W = torch.full((256, 144), 1e38, device="cuda")
    W[3, 5], W[130, 7], W[255, 143] = top, -top, top
    q, s = torch.zeros(W.shape, device="cuda").to(E4M3), torch.zeros(2, 2, device="cuda")
    lib.prepare_linear_fp8(W, q, s)
    lib.sync_status()
    want_s = torch.tensor([[top, 1e38], [top, top]], device="cuda").to(F64) / 448.0
    assert torch.equal(s, want_s.float())
    v = W.to(F64) / s.to(F64).repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :144]
    assert torch.equal(q.float().to(F64), P.e4m3_round(v))
    for bad in (math.nan, math.inf, -math.inf):
        for at in ((0, 0), (255, 143), (7, 130)):
            V = W.clone()
            V[at] = bad
            lib.prepare_linear_fp8(V, q, s)
            with pytest.raises(lib.FmError) as e:
                lib.sync_status()
            assert e.value.status == 5
