"""The token loop's operators at the borders of their definitions: exact ties of
codes, the largest weights, candidates of different beams that lie close."""
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


# ------------------------------------------------------------------ beam selection
def check(lib, logits, scores, n_out, finished=None, eos=-1, ws=None):
    B, k, V = logits.shape
    out = torch.full((B, n_out), 77.0, device="cuda")
    par, tok = (torch.full((B, n_out), 77, device="cuda", dtype=torch.int32) for _ in range(2))
    fin = torch.full((B, n_out), 77, device="cuda", dtype=torch.uint8)
    if ws is None:
        ws = torch.full((lib.beam_workspace_bytes(B, k, V, n_out),), 255, device="cuda", dtype=torch.uint8)
    lib.beam_select(logits, scores, out, par, tok, ws, finished=finished, out_finished=fin, eos=eos)
    lib.sync_status()
    want = P.beam(logits.cpu(), scores.cpu(), None if finished is None else finished.cpu(), eos, n_out)
    assert torch.equal(par.cpu().long(), want[1])
    assert torch.equal(tok.cpu().long(), want[2])
    assert torch.equal(fin.cpu(), want[3])
    w, got = want[0], out.cpu().to(F64)
    live = w > -torch.inf
    assert torch.equal(got > -torch.inf, live)
    # c is rounded once to fp32 after a log sum whose arguments are rounded three
    # times in fp32 (2.25 * 2^-24 of ln V on average), whose exponentials are off
    # by 2^-22, and of which 16 at a time are added in fp32 (15 * 2^-24)
    tol = w.abs() * 2.0 ** -24 + (2.25 * math.log(V) + 20) * 2.0 ** -24
    assert bool(((got - w).abs()[live] <= tol[live]).all())
    return got, w


def row(V, first, d, n):
    """One logit of 0 at `first` and n of -d behind it, the rest masked."""
    l = torch.full((V,), -math.inf)
    l[first] = 0.0
    l[first + 1:first + 1 + n] = -d
    return l


def lse(l):
    return float(torch.logsumexp(l.to(F64), 0))


def near_pair(V, d1, n1, d2, margin):
    """Two rows and scores whose best candidates differ by `margin` (beam 1's is
    worth more where it is positive)."""
    a = row(V, 5, d1, n1)
    b = row(V, 7, d2, round(n1 * math.exp(d2 - d1)))
    return torch.stack([a, b]), torch.tensor([0.0, lse(b) - lse(a) + margin])


PAIRS = [(9.5, 60000, 5.0), (5.0, 600, 9.5), (13.0, 99000, 10.25), (10.25, 6000, 13.0), (7.0, 90000, 2.75),
         (11.5, 99000, 0.5)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_out", [1, 2, 5])
def test_select_between_close_beams(lib, n_out, dtype):
    """Candidates of two beams that differ by less than fp32 tells apart are taken
    in the order of their 64-bit values; alone and in a batch."""
    V, cases = 100003, []
    for d1, n1, d2 in PAIRS:
        for m in (3e-8, 1e-7, 4e-7, 2e-6):
            cases += [near_pair(V, d1, n1, d2, m), near_pair(V, d1, n1, d2, -m)]
    logits = torch.stack([c[0] for c in cases]).to("cuda", dtype)
    scores = torch.stack([c[1] for c in cases]).float().cuda()
    check(lib, logits, scores, n_out)
    for b in range(0, len(cases), 5):
        check(lib, logits[b:b + 1].clone(), scores[b:b + 1].clone(), n_out)


def test_select_among_many_close_beams(lib):
    """Eight beams in a tangle, an ended beam among them, and one beam's second
    candidate beside another's first."""
    V, k, g = 30011, 8, torch.Generator().manual_seed(3)
    logits, scores = torch.empty(4, k, V), torch.empty(4, k)
    for b in range(4):
        for j in range(k):
            d = 2.0 + 9.0 * float(torch.rand((), generator=g))
            l = row(V, 3 * j, d, min(20000, round(0.3 * math.exp(d))))
            l[V - 1 - j] = -1e-7 * (j + 1)
            logits[b, j] = l
            scores[b, j] = lse(l) - 0.5 + 1e-6 * (float(torch.rand((), generator=g)) - 0.5)
    scores[1:] += torch.tensor([0.0, -3.0, -40.0])[:, None]
    fin = torch.zeros(4, k, dtype=torch.uint8)
    fin[0, 2] = fin[2, 5] = 1
    scores[0, 2], scores[2, 5] = -0.5, -3.5
    for n_out in (1, 3, 8, 16):
        check(lib, logits.cuda(), scores.cuda(), n_out, fin.cuda(), 11)
        check(lib, logits[:1].cuda(), scores[:1].cuda(), n_out, fin[:1].cuda(), 11)


@pytest.mark.parametrize("margin", [-1e-6, -2e-7, 2e-7, 1e-6])
def test_select_with_an_ended_beam_between_two_close_ones(lib, margin):
    """The one candidate taken, an ended beam's below it, and a third beam's that
    only the 64-bit sums place."""
    V = 100003
    for d1, n1, d2 in PAIRS:
        l, s = near_pair(V, d1, n1, d2, margin)
        logits = torch.full((1, 3, V), -1.0)
        logits[0, 0], logits[0, 2] = l[0], l[1]
        first = -lse(l[0])
        for below in (0.0, 1e-6, 2.7e-6, 4e-6):
            scores = torch.tensor([[0.0, first - below, s[1]]])
            fin = torch.tensor([[0, 1, 0]], dtype=torch.uint8)
            for n_out in (1, 2, 3):
                check(lib, logits.cuda(), scores.float().cuda(), n_out, fin.cuda(), 9)


def test_select_between_close_beams_with_masks_and_odd_rows(lib):
    """The same with NaN and infinite logits in the rows and rows of odd strides."""
    V = 20011
    wide = torch.full((2, 2, V + 5), 3.0)
    scores = torch.zeros(2, 2)
    for b, m in enumerate((1e-7, -1e-7)):
        wide[b, :, :V], scores[b] = near_pair(V, 9.0, 15000, 4.5, m)
    wide[:, :, 15:18] = math.nan
    wide[:, 0, 18] = -math.inf
    for b, m in enumerate((1e-7, -1e-7)):
        l = torch.nan_to_num(wide[b, :, :V].to(F64), nan=-math.inf, neginf=-math.inf)
        scores[b, 1] = scores[b, 0] + lse(l[1]) - lse(l[0]) + m
    check(lib, wide.cuda()[:, :, :V], scores.cuda(), 4)


def test_select_with_one_workspace_for_a_shrinking_batch(lib):
    """A workspace sized for the largest batch serves every smaller one."""
    g = torch.Generator(device="cuda").manual_seed(5)
    V, n = 50000, 8
    ws = torch.empty(lib.beam_workspace_bytes(13, 2, V, n), device="cuda", dtype=torch.uint8)
    assert lib.beam_workspace_bytes(1, 1, 1, 1) > 0
    logits = torch.randn(13, 2, V, device="cuda", generator=g)
    scores = -torch.rand(13, 2, device="cuda", generator=g)
    for B in (13, 12, 11, 10, 4, 1):
        check(lib, logits[:B], scores[:B], n, ws=ws)
