"""The token loop's operators on the GPU against their 64-bit plain forms:
residual RMSNorm to 8-bit codes, the block-scaled e4m3 product, embedding rows,
beam selection, state reordering, and all of them together in DeviceLM."""
import math

import numpy as np
import pytest

from quantized_state_space_mamba2_b200 import synth as S

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


# ------------------------------------------------------------------ norm
def check_norm(lib, x, w, residual, kind, sum_out=None, eps=1e-5):
    M, K = x.shape
    q = torch.full((M, K), 1, device="cuda").to(E4M3 if kind == "e4m3" else torch.int8)
    s = torch.full((M, P.blocks(K)) if kind == "e4m3" else (M,), -1.0, device="cuda")
    r, codes, scales, sure = P.norm(x, residual, w, eps, kind)  # before an in-place call
    lib.add_norm_quant(x, w, q, s, residual=residual, sum_out=sum_out, eps=eps)
    lib.sync_status()
    # exact: sums and statistics in 64 bits on both sides; a code within 2^-44
    # of a border (none is expected) may be either neighbour
    assert torch.equal(s, scales)
    assert bool(((q.float().to(F64) == codes) | (sure == 0)).all())
    if sum_out is not None:
        assert torch.equal(sum_out, r)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 112), (5, 128), (2, 144), (257, 768), (64, 2560),
                                 (3, 5136), (2, 8192), (2, 16384), (1, 512), (1, 528)])
def test_norm(lib, M, K, dtype, kind):
    g = gen(M * 31 + K)
    x = randn(g, M, K)
    x[:, ::97] *= 60.0
    w = 1.0 + 0.2 * randn(g, K)
    check_norm(lib, x.to(dtype), w, None, kind)
    r = 2.0 * randn(g, M, K)
    check_norm(lib, x.to(dtype), w, r, kind, sum_out=torch.empty(M, K, device="cuda"))
    check_norm(lib, x.to(dtype), w, r, kind, sum_out=r)  # the residual stream in place


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_norm_strides_zeros_magnitudes(lib, kind):
    g = gen(4)
    K, M = 400, 9
    wide = randn(g, M, 3, K + 32)
    x, res = wide[:, 1, 4:K + 4], wide[:, 2, :K]
    buf = torch.full((M, K + 4), 7.0, device="cuda")
    w = 1.0 + 0.2 * randn(g, K)
    check_norm(lib, x, w, res, kind, sum_out=buf[:, :K])
    assert bool((buf[:, K:] == 7.0).all())
    check_norm(lib, wide.view(-1, K + 32)[::3][:, :K].bfloat16(), w, None, kind)
    # zero rows, a zero block, zero weights, the largest and smallest rows
    x = randn(g, 8, K)
    x[0] = 0.0
    x[1, 128:256] = 0.0
    x[2] *= 1e37
    x[3] *= 1e-30
    x[4] *= 1e-44  # subnormal
    x[5, 1:] = 0.0
    x[6] = 3.0  # every element is the maximum
    w[:128] = 0.0
    check_norm(lib, x, w, None, kind)
    check_norm(lib, x, w, None, kind, eps=0.25)
    check_norm(lib, x[:, :16].contiguous(), torch.full((16,), 1e-34, device="cuda"), None, kind)
    # mean square 1, weight 1: arguments on exact borders of the int8 codes
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, 63.5, -126.5] + [0.0] * 10], device="cuda")
    check_norm(lib, x, torch.ones(16, device="cuda"), None, kind, eps=1e-30)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_norm_reports_nonfinite(lib, bad):
    x = torch.ones(4, 256, device="cuda")
    x[2, 17] = bad
    q = torch.zeros(4, 256, device="cuda", dtype=torch.int8)
    s = torch.zeros(4, device="cuda")
    lib.add_norm_quant(x, torch.ones(256, device="cuda"), q, s)
    with pytest.raises(lib.FmError) as e:
        lib.sync_status()
    assert e.value.status == 5
    lib.sync_status()  # read and cleared
    assert bool((q[[0, 1, 3]] == 127).all())  # the other rows are whole


# ------------------------------------------------------------------ prepared weights, product
@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (129, 144), (300, 768), (77, 2560)])
def test_prepare_linear_fp8(lib, N, K):
    g = gen(N + K)
    W = 0.02 * randn(g, N, K)
    W[0, 0] = 5.0
    if N > 128:
        W[128:] = 0.0
    q = torch.empty(N, K, device="cuda", dtype=E4M3)
    s = torch.empty(P.blocks(N), P.blocks(K), device="cuda")
    lib.prepare_linear_fp8(W, q, s)
    lib.sync_status()
    pad = torch.zeros(P.blocks(N) * 128, P.blocks(K) * 128, device="cuda", dtype=F64)
    pad[:N, :K] = W
    b = pad.view(P.blocks(N), 128, P.blocks(K), 128)
    want_s = (b.abs().amax((1, 3)) / 448.0).float()
    assert torch.equal(s, want_s)
    sd = want_s.to(F64)[:, None, :, None]
    v = torch.where(sd > 0, b / sd.clamp_min(2.0 ** -140), 0.0).reshape(pad.shape)[:N, :K]
    assert torch.equal(q.float().to(F64), P.e4m3_round(v))


def product_case(g, M, N, K, spread=1.0):
    """Random codes over e4m3's whole range and positive scales."""
    def codes(r):
        c = torch.randint(0, 256, (r, K), device="cuda", generator=g, dtype=torch.int32)
        c = torch.where((c & 127) == 127, c - 1, c)  # 0x7f, 0xff are NaN
        return c.to(torch.uint8).view(E4M3)

    def scales(r):
        return torch.exp(spread * randn(g, r, P.blocks(K))) * 2.0 ** -9

    return codes(M), scales(M), codes(N), scales(P.blocks(N))


def check_product(lib, a, sa, w, sw, y):
    M, K, N = a.shape[0], a.shape[1], w.shape[0]
    lib.fp8_gemm(a, sa, w, sw, y)
    lib.sync_status()
    da, dw = P.dequant_rows(a, sa), P.dequant_blocks(w, sw)
    want, size = da @ dw.t(), da.abs() @ dw.abs().t()
    # the 128 exact products of a block are summed in fp32, rounded or cut
    # (128 * 2^-23); the block's scale product and its product with the sum are
    # rounded, and up to K / 128 block terms added (each 2^-24); every error is
    # relative to sum |a w|.  The result is rounded once to Y's type.
    tol = (128 * 2.0 ** -23 + (P.blocks(K) + 3) * 2.0 ** -24) * size
    tol = tol + (want.abs() + tol) * torch.finfo(y.dtype).eps / 2
    assert bool(((y.to(F64) - want).abs() <= tol).all())
    # the errors do not add up in one direction: their rms is far below that bound
    if M * N >= 64 and y.dtype == torch.float32:
        rms = lambda t: float(t.square().mean().sqrt())
        assert rms(y.to(F64) - want) <= 2e-6 * rms(want)


SIZES = [(1, 1, 16), (1, 7, 128), (2, 129, 144), (4, 1001, 768), (15, 33, 256), (16, 128, 128),
         (17, 300, 400), (33, 513, 1040), (64, 2000, 2560), (65, 257, 384), (100, 640, 512),
         (128, 1000, 768), (129, 255, 640), (200, 999, 272), (257, 1537, 1536), (300, 128, 16),
         (1000, 130, 32), (513, 4097, 144), (7, 300, 8320), (100, 140, 16400), (130, 140, 8336),
         (20, 20000, 8448)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(lib, M, N, K, dtype):
    g = gen(M * 7 + N * 3 + K)
    check_product(lib, *product_case(g, M, N, K), torch.empty(M, N, device="cuda", dtype=dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,ldy", [(5, 100, 104), (5, 100, 131), (70, 200, 257), (300, 260, 264),
                                     (300, 131, 145)])
def test_product_into_strided_rows(lib, M, N, ldy, dtype):
    g = gen(ldy)
    buf = torch.full((M, ldy), 3.0, device="cuda", dtype=dtype)
    check_product(lib, *product_case(g, M, N, 256), buf[:, :N])
    assert bool((buf[:, N:] == 3.0).all())


def test_product_is_the_same_every_time_and_rows_are_independent(lib):
    g = gen(9)
    a, sa, w, sw = product_case(g, 200, 700, 640)
    y = torch.empty(200, 700, device="cuda")
    lib.fp8_gemm(a, sa, w, sw, y)
    again = torch.empty_like(y)
    lib.fp8_gemm(a, sa, w, sw, again)
    assert torch.equal(y, again)
    # a zero scale makes its block vanish; a NaN code reaches its own row only
    sa2 = sa.clone()
    sa2[3, 2] = 0.0
    a2 = a.clone()
    a2.view(torch.uint8)[5, 11] = 0x7F
    lib.fp8_gemm(a2, sa2, w, sw, again)
    lib.sync_status()
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[[3, 5]] = False
    assert torch.equal(y[keep], again[keep])
    assert bool(again[5].isnan().all()) and bool(again[3].isfinite().all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K,ldy", [(2500, 2700, 400, 2700), (4001, 1301, 144, 1301), (300, 9601, 16, 9601),
                                       (8200, 700, 2560, 704), (257, 19000, 640, 19013),
                                       (20000, 130, 128, 136)])
def test_product_on_pairs_of_ctas(lib, M, N, K, ldy, dtype):
    g = gen(M + N)
    buf = torch.full((M, ldy), 3.0, device="cuda", dtype=dtype)
    check_product(lib, *product_case(g, M, N, K, 0.3), buf[:, :N])
    assert bool((buf[:, N:] == 3.0).all())


def test_product_large(lib):
    # more tiles than SMs in both directions, and K of 20 blocks
    g = gen(12)
    check_product(lib, *product_case(g, 1200, 3100, 2560, 0.3), torch.empty(1200, 3100, device="cuda"))
    check_product(lib, *product_case(g, 48, 50000, 768, 0.3), torch.empty(48, 50000, device="cuda"))


@pytest.mark.parametrize("M,N,K", [(5, 1000, 768), (100, 5000, 400), (300, 3000, 2560), (2500, 2700, 640)])
def test_product_reports_a_wait_that_gave_up(lib, M, N, K):
    """Loads that are never issued: the waits run out after 20 ms, the call ends
    and says so, and the next one is right (every kernel variant)."""
    g = gen(K)
    case = product_case(g, M, N, K, 0.3)
    y = torch.empty(M, N, device="cuda")
    lib.sync_status()
    lib.set_fault_injection(lib.STALL_GEMM, 20_000_000)
    try:
        lib.fp8_gemm(*case, y)
        torch.cuda.synchronize()
    finally:
        lib.set_fault_injection(0, 0)
    with pytest.raises(lib.FmError) as e:
        lib.sync_status()
    assert e.value.status == 6
    check_product(lib, *case, y)


# ------------------------------------------------------------------ embedding rows
@pytest.mark.parametrize("kind", ["fp32", "bf16", "e4m3"])
@pytest.mark.parametrize("M,V,K", [(1, 1, 16), (7, 130, 144), (64, 1000, 2560), (300, 257, 768),
                                   (2, 5, 4112)])
def test_embed(lib, M, V, K, kind):
    g = gen(M + V + K)
    t, ts = randn(g, V, K), None
    if kind == "e4m3":
        q = torch.empty(V, K, device="cuda", dtype=E4M3)
        ts = torch.empty(P.blocks(V), P.blocks(K), device="cuda")
        lib.prepare_linear_fp8(t, q, ts)
        t = q
    elif kind == "bf16":
        t = t.bfloat16()
    ids = torch.randint(-1, V, (M,), device="cuda", generator=g, dtype=torch.int32)
    ids[0] = V - 1
    buf = torch.full((M, K + 16), 5.0, device="cuda")
    lib.embed_rows(ids, t, buf[:, :K], table_s=ts, scale=3.7)
    lib.sync_status()
    at = ids.long().clamp_min(0)
    want = t[at].float()
    if ts is not None:
        want = want * ts[at // 128].repeat_interleave(128, 1)[:, :K]
    want = torch.where(ids[:, None] >= 0, want * torch.tensor(3.7, device="cuda"), 0.0)
    assert torch.equal(buf[:, :K], want) and bool((buf[:, K:] == 5.0).all())


def test_a_stream_argument(lib):
    """stream= queues the call there: behind what that stream has been given."""
    side = torch.cuda.Stream()
    t = torch.zeros(8, 4096, device="cuda")
    ids = torch.arange(8, device="cuda", dtype=torch.int32)
    x = torch.full((8, 4096), -1.0, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for v in range(200):
            t.fill_(float(v))
    lib.embed_rows(ids, t, x, stream=side)
    side.synchronize()
    assert bool((x == 199.0).all())


@pytest.mark.parametrize("bad", [-2, 40, 2 ** 31 - 1, -2 ** 31])
def test_embed_reports_bad_ids(lib, bad):
    t = torch.ones(40, 32, device="cuda")
    x = torch.full((3, 32), 9.0, device="cuda")
    lib.embed_rows(torch.tensor([1, bad, 39], device="cuda", dtype=torch.int32), t, x)
    with pytest.raises(lib.FmError) as e:
        lib.sync_status()
    assert e.value.status == 9
    assert bool((x[1] == 0).all()) and bool((x[[0, 2]] == 1).all())


# ------------------------------------------------------------------ beam selection
def select(lib, logits, scores, n_out, finished=None, eos=-1):
    B, k, V = logits.shape
    out = torch.full((B, n_out), 77.0, device="cuda")
    par, tok = (torch.full((B, n_out), 77, device="cuda", dtype=torch.int32) for _ in range(2))
    fin = torch.full((B, n_out), 77, device="cuda", dtype=torch.uint8)
    ws = torch.full((lib.beam_workspace_bytes(B, k, V, n_out),), 255, device="cuda", dtype=torch.uint8)
    lib.beam_select(logits, scores, out, par, tok, ws, finished=finished, out_finished=fin, eos=eos)
    lib.sync_status()
    return out, par, tok, fin


def check_select(lib, logits, scores, n_out, finished=None, eos=-1):
    out, par, tok, fin = (t.cpu() for t in select(lib, logits, scores, n_out, finished, eos))
    want = P.beam(logits.cpu(), scores.cpu(), None if finished is None else finished.cpu(), eos, n_out)
    assert torch.equal(par.long(), want[1])
    assert torch.equal(tok.long(), want[2])
    assert torch.equal(fin, want[3])
    w, got = want[0], out.to(F64)
    live = w > -torch.inf
    assert torch.equal(got > -torch.inf, live)
    # c is rounded once to fp32; exp in fp32 (2 ulp) and its argument's rounding
    # (2^-24 of at most about 100) move the sum, so lse, by less than 2^-17
    tol = w.abs() * 2.0 ** -24 + 2.0 ** -17
    assert bool(((got - w).abs()[live] <= tol[live]).all())


SELECT = [(1, 1, 1, 1), (2, 3, 2, 5), (1, 4, 7, 4), (3, 2, 31, 32), (2, 32, 33, 32), (1, 1, 257, 8),
          (2, 5, 1000, 3), (1, 4, 32001, 4), (3, 8, 50000, 8), (1, 16, 4099, 16), (1, 1, 100003, 1),
          (1, 2, 8191, 32), (1, 3, 8193, 7)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,k,V,n", SELECT)
def test_select(lib, B, k, V, n, dtype):
    g = gen(B + 10 * k + V + n)
    logits = 2.5 * randn(g, B, k, V)
    scores = -torch.rand(B, k, device="cuda", generator=g).cumsum(1) - 3.0
    check_select(lib, logits.to(dtype), scores, n)
    logits[:, :, torch.rand(V, device="cuda", generator=g) < 0.4] = -math.inf
    fin = (torch.rand(B, k, device="cuda", generator=g) < 0.4).to(torch.uint8)
    check_select(lib, logits.to(dtype), scores, n, fin, eos=V // 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 300, 20011])
def test_select_orders_ties_and_masks(lib, V, dtype):
    z = lambda *s: torch.zeros(*s, device="cuda", dtype=dtype)
    sc = torch.zeros(2, 3, device="cuda")
    check_select(lib, z(2, 3, V), sc, 4)  # every candidate equal: the lowest ones
    l = z(2, 3, V)
    l[:, :, V // 2:] = 1.0  # many ties at the top
    check_select(lib, l, sc, 8)
    check_select(lib, -l, sc, 8)  # -0 beside 0
    up = torch.arange(V, device="cuda").to(dtype).expand(2, 3, V).contiguous()
    check_select(lib, up / V, sc, 5)  # ascending: every value is a new best
    check_select(lib, -up / V, sc, 5)
    # empty rows, an empty entry, NaN, infinities, dead and NaN scores
    l = torch.randn(2, 3, V, device="cuda", generator=gen(V)).to(dtype)
    l[0, 1] = -math.inf
    l[1] = -math.inf
    check_select(lib, l, sc, 6)
    l = torch.randn(2, 3, V, device="cuda", generator=gen(V + 1)).to(dtype)
    l[0, 0, 1] = math.nan
    l[0, 1, :] = math.nan
    l[1, 2, 3] = math.inf
    l[1, 0, 2] = torch.finfo(dtype).min
    s = sc.clone()
    s[0, 2] = -math.inf
    s[1, 0] = math.nan
    s[1, 1] = -1.0
    check_select(lib, l, s, 6)
    l = torch.full((2, 3, V), torch.finfo(dtype).min, device="cuda", dtype=dtype)
    check_select(lib, l, s, 4)  # the type's lowest value is a value, not a mask
    l[:, :, 2] = math.inf
    check_select(lib, l, s, 4)


def test_select_fewer_candidates_than_slots(lib):
    l = torch.full((2, 2, 40), -math.inf, device="cuda")
    l[0, 1, 7] = 0.5
    sc = torch.tensor([[-1.0, -2.0], [-1.0, -math.inf]], device="cuda")
    check_select(lib, l, sc, 5)
    check_select(lib, l, sc, 5, torch.tensor([[1, 0], [1, 1]], device="cuda", dtype=torch.uint8), eos=0)


def test_select_strides_in_place_and_determinism(lib):
    g = gen(2)
    B, k, V = 3, 4, 5003
    wide = 2.0 * randn(g, B, k, V + 13)
    l = wide[:, :, 4:V + 4]
    sc = -torch.rand(B, k, device="cuda", generator=g)
    check_select(lib, l, sc, 4)
    fin = (torch.rand(B, k, device="cuda", generator=g) < 0.5).to(torch.uint8)
    want = select(lib, l, sc, k, fin, 9)
    s2, f2 = sc.clone(), fin.clone()
    par, tok = (torch.empty(B, k, device="cuda", dtype=torch.int32) for _ in range(2))
    ws = torch.empty(lib.beam_workspace_bytes(B, k, V, k), device="cuda", dtype=torch.uint8)
    lib.beam_select(l, s2, s2, par, tok, ws, finished=f2, out_finished=f2, eos=9)
    lib.sync_status()
    assert all(torch.equal(a, b) for a, b in zip((s2, par, tok, f2), want))


# ------------------------------------------------------------------ state reordering
def check_reorder(lib, shapes, dtypes, B, beams, g, src_beams=None, parent=None):
    sb = beams if src_beams is None else src_beams
    src = [torch.randint(-100, 100, (B * sb, *s), device="cuda", generator=g).to(t)
           for s, t in zip(shapes, dtypes)]
    if parent is None:
        parent = torch.randint(0, sb, (B, beams), device="cuda", generator=g, dtype=torch.int32)
    at = (torch.arange(B, device="cuda")[:, None] * sb + parent).view(-1)
    want = [t[at] for t in src]
    dst = src if src_beams is None else [torch.empty(B * beams, *t.shape[1:], device="cuda",
                                                     dtype=t.dtype) for t in src]
    lib.reorder_rows(lib.RowSet(dst, None if src_beams is None else src), parent, src_beams=src_beams)
    lib.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(dst, want))


@pytest.mark.parametrize("B,beams", [(1, 1), (1, 2), (3, 4), (2, 7), (5, 8), (2, 16), (1, 32)])
def test_reorder(lib, B, beams):
    g = gen(B * 100 + beams)
    shapes = [(3, 512), (4, 64, 128), (7,), (3,), (5, 3, 3), (1024, 9)]
    dtypes = [torch.int8, torch.int32, torch.int32, torch.int8, torch.int16, torch.float32]
    check_reorder(lib, shapes, dtypes, B, beams, g)
    check_reorder(lib, shapes, dtypes, B, beams, g, src_beams=1)
    check_reorder(lib, shapes, dtypes, B, beams, g, src_beams=min(beams + 3, 32))
    ident = torch.arange(beams, device="cuda", dtype=torch.int32).expand(B, beams).contiguous()
    check_reorder(lib, shapes, dtypes, B, beams, g, parent=ident)
    check_reorder(lib, shapes, dtypes, B, beams, g, parent=ident.flip(1).contiguous())
    check_reorder(lib, shapes, dtypes, B, beams, g, parent=ident.roll(1, 1).contiguous())
    check_reorder(lib, shapes, dtypes, B, beams, g, parent=torch.full_like(ident, beams - 1))


def test_reorder_many_buffers(lib):
    # more than one launch holds, of three unit sizes in turn
    n = 300
    check_reorder(lib, [(48 + (i % 3),) for i in range(n)],
                  [(torch.int32, torch.int8)[i % 2] for i in range(n)], 2, 5, gen(3))


@pytest.mark.parametrize("bad", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_reorder_reports_bad_parents(lib, bad):
    t = torch.arange(8 * 64, device="cuda", dtype=torch.int32).view(8, 64)
    old = t.clone()
    parent = torch.tensor([[1, bad, 0, 3], [3, 2, 1, 0]], device="cuda", dtype=torch.int32)
    lib.reorder_rows(lib.RowSet([t]), parent)
    with pytest.raises(lib.FmError) as e:
        lib.sync_status()
    assert e.value.status == 9
    assert torch.equal(t, old[[1, 1, 0, 3, 7, 6, 5, 4]])


# ------------------------------------------------------------------ streams and graphs
def test_another_stream_and_a_replayed_graph(lib):
    """The whole chain on a side stream and in one captured graph gives the bits
    of the calls on the current stream; a replay sees new inputs."""
    g = gen(21)
    B, k, V, K = 2, 3, 1003, 512
    W = 0.1 * randn(g, V, K)
    t = torch.empty(V, K, device="cuda", dtype=E4M3)
    ts = torch.empty(P.blocks(V), P.blocks(K), device="cuda")
    lib.prepare_linear_fp8(W, t, ts)
    w = torch.ones(K, device="cuda")

    def buffers():
        e = lambda *s, dtype=torch.float32: torch.zeros(*s, device="cuda", dtype=dtype)
        return dict(ids=e(B * k, dtype=torch.int32), x=e(B * k, K), q=e(B * k, K, dtype=torch.int8).view(E4M3),
                    s=e(B * k, P.blocks(K)), y=e(B * k, V), sc=e(B, k), par=e(B, k, dtype=torch.int32),
                    tok=e(B, k, dtype=torch.int32), state=e(B * k, 64, dtype=torch.int32),
                    ws=e(lib.beam_workspace_bytes(B, k, V, k), dtype=torch.uint8))

    def chain(c, rows):
        lib.embed_rows(c["ids"], t, c["x"], ts, 5.0)
        lib.add_norm_quant(c["x"], w, c["q"], c["s"], residual=c["x"], sum_out=c["x"])
        lib.fp8_gemm(c["q"], c["s"], t, ts, c["y"])
        lib.beam_select(c["y"].view(B, k, V), c["sc"], c["sc"], c["par"], c["tok"], c["ws"])
        lib.reorder_rows(rows, c["par"])

    def fill(c, seed):
        h = gen(seed)
        c["ids"].copy_(torch.randint(0, V, (B * k,), device="cuda", generator=h, dtype=torch.int32))
        c["sc"].copy_(-torch.rand(B, k, device="cuda", generator=h))
        c["state"].copy_(torch.randint(0, 99, (B * k, 64), device="cuda", generator=h, dtype=torch.int32))

    def snap(c):
        return {n: v.clone() for n, v in c.items() if n != "ws"}

    plain, want = buffers(), {}
    rows = lib.RowSet([plain["state"]])
    for seed in (1, 2):
        fill(plain, seed)
        chain(plain, rows)
        want[seed] = snap(plain)
    lib.sync_status()

    def same(c, seed):
        return all(torch.equal(c[n].view(torch.uint8) if v.dtype == E4M3 else c[n],
                               v.view(torch.uint8) if v.dtype == E4M3 else v)
                   for n, v in want[seed].items())

    side = torch.cuda.Stream()
    a, b = buffers(), buffers()
    fill(a, 1)
    ra, rb = lib.RowSet([a["state"]]), lib.RowSet([b["state"]])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        chain(a, ra)
    side.synchronize()
    assert same(a, 1)
    graph = torch.cuda.CUDAGraph()
    fill(b, 1)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chain(b, rb)
    for seed in (2, 1, 2):
        fill(b, seed)
        graph.replay()
        torch.cuda.synchronize()
        assert same(b, seed)
    lib.sync_status()


def test_two_streams_at_once(lib):
    """Two chains of calls on two streams, each with its own buffers, give the
    bits of one alone."""
    g = gen(31)
    K, V, B, k = 768, 9001, 4, 4
    t = torch.empty(V, K, device="cuda", dtype=E4M3)
    ts = torch.empty(P.blocks(V), P.blocks(K), device="cuda")
    lib.prepare_linear_fp8(0.1 * randn(g, V, K), t, ts)
    w, x = torch.ones(K, device="cuda"), randn(g, 700, K)

    def chain(reps):
        e = lambda *s, dtype=torch.float32: torch.zeros(*s, device="cuda", dtype=dtype)
        q, s = e(700, K, dtype=torch.int8).view(E4M3), e(700, P.blocks(K))
        y, z, sc = e(700, V), e(16, V), e(B, k)
        par, tok = e(B, k, dtype=torch.int32), e(B, k, dtype=torch.int32)
        ws = e(lib.beam_workspace_bytes(B, k, V, k), dtype=torch.uint8)
        state = torch.arange(B * k * 4096, device="cuda", dtype=torch.int32).view(B * k, 4096)
        rows = lib.RowSet([state])
        for _ in range(reps):
            lib.add_norm_quant(x, w, q, s)
            lib.fp8_gemm(q, s, t, ts, y)
            lib.fp8_gemm(q[:16], s[:16], t, ts, z)
            lib.beam_select(z.view(B, k, V), sc, sc, par, tok, ws)
            lib.reorder_rows(rows, par)
        return y, z, sc, par, tok, state

    want = chain(6)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        with torch.cuda.stream(st):
            got.append(chain(6))
    torch.cuda.synchronize()
    lib.sync_status()
    assert all(torch.equal(a, b) for one in got for a, b in zip(one, want))


def test_offsets_past_32_bits(lib):
    g = gen(41)
    # a table of more than 2^31 elements
    V, K = 140001, 16384
    t = torch.zeros(V, K, device="cuda", dtype=torch.bfloat16)
    t[-1] = randn(g, K).bfloat16()
    t[7] = randn(g, K).bfloat16()
    x = torch.empty(3, K, device="cuda")
    lib.embed_rows(torch.tensor([V - 1, 7, V - 1], device="cuda", dtype=torch.int32), t, x)
    assert torch.equal(x, t[[V - 1, 7, V - 1]].float())
    del t
    # a product with as many outputs, and one with a long row stride
    M, N = 66001, 33000
    a, sa, w, sw = product_case(g, M, N, 16, 0.3)
    y = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    lib.fp8_gemm(a, sa, w, sw, y)
    lib.sync_status()
    want = P.dequant_rows(a[-70:], sa[-70:]) @ P.dequant_blocks(w, sw).t()
    tol = (want.abs() + 1e-3 * want.abs().mean()) * 2.0 ** -8
    assert bool(((y[-70:].to(F64) - want).abs() <= tol).all())
    del y
    wide = torch.zeros(40, 60_000_000, device="cuda", dtype=torch.bfloat16)
    lib.fp8_gemm(a[:40], sa[:40], w[:500], sw[:4], wide[:, :500])
    lib.sync_status()
    want = P.dequant_rows(a[:40], sa[:40]) @ P.dequant_blocks(w[:500], sw[:4]).t()
    assert bool(((wide[:, :500].to(F64) - want).abs() <= (want.abs() + 1e-3 * want.abs().mean()) * 2.0 ** -8).all())
    # logits of as many elements
    del wide
    l = torch.zeros(75, 6, 5_000_003, device="cuda", dtype=torch.bfloat16)
    l[74, 5, 5_000_002] = 9.0
    l[74, 2, 4_999_000] = 8.0
    sc = torch.zeros(75, 6, device="cuda")
    out = select(lib, l, sc, 3)
    assert out[1][74, :2].tolist() == [5, 2] and out[2][74, :2].tolist() == [5_000_002, 4_999_000]
    assert out[1][73].tolist() == [0, 0, 0] and out[2][73].tolist() == [0, 1, 2]


# ------------------------------------------------------------------ all of them together
@pytest.fixture(scope="module")
def model(lib):
    from quantized_state_space_mamba2_b200.model import DeviceLM
    shape = S.MixerShape(d_model=256, d_inner=512, headdim=64, d_state=128)
    V = 301
    rng = np.random.default_rng(5)
    emb = rng.normal(0, 0.3, (V, 256)).astype(np.float32)
    head = rng.normal(0, 0.08, (V, 256)).astype(np.float32)
    lm = DeviceLM([S.layer_params(shape, 60 + l) for l in range(3)], shape, emb,
                  1.0 + 0.1 * rng.normal(size=256).astype(np.float32), head=head, embed_scale=4.0)
    ids = torch.from_numpy(rng.integers(0, V, (2, 64)).astype(np.int32)).cuda()
    lm.calibrate(ids)
    return lm, V, rng


def plain_logits(lm, ids):
    """Logits after ids [B, T], from the stack's rows of the whole sequences and
    the plain norm and head."""
    x = lm.embed(ids)
    lm.stack.prefill_(x)
    r, codes, s, _ = P.norm(x[:, -1], None, lm.norm_w, 1e-5, "e4m3")
    return (P.dequant_rows(codes.float(), s) @ P.dequant_blocks(lm.head, lm.head_s).t()).cpu()


@pytest.mark.parametrize("eos", [-1, 7])
@pytest.mark.parametrize("beams", [1, 4])
def test_beam_search_against_whole_sequences(lib, model, beams, eos):
    lm, V, rng = model
    B, T, steps = 2, 37, 8
    ids = torch.from_numpy(np.random.default_rng(beams).integers(0, V, (B, T)).astype(np.int32)).cuda()
    tokens, scores = lm.beam_search(ids, beams, steps, eos)
    lib.sync_status()
    # the plain search keeps no state: every step runs each beam's whole sequence
    hist = [[[] for _ in range(1)] for _ in range(B)]
    sc = torch.zeros(B, 1)
    fin = None
    for t in range(steps):
        k = sc.shape[1]
        l = torch.zeros(B, k, V, dtype=F64)
        for b in range(B):
            for j in range(k):
                seq = torch.cat([ids[b], torch.tensor(hist[b][j], device="cuda", dtype=torch.int32)])
                l[b, j] = plain_logits(lm, seq[None])[0]
        v, par, tok, nf = P.beam(l, sc, fin, eos, beams)
        hist = [[hist[b][int(par[b, j])] + [int(tok[b, j])] for j in range(beams)] for b in range(B)]
        sc, fin = v, (nf if eos >= 0 else None)
    assert tokens.cpu().tolist() == hist
    # per step: logits (fp32 sums of 256 products), lse and the score's rounding
    assert bool(((scores.cpu().to(F64) - sc).abs() <= steps * (2.0 ** -17 + 2.0 ** -15)).all())


def test_decode_matches_prefill_logits(lib, model):
    """A prompt in one prefill, and its last tokens one by one, give the same
    logits bits; in a captured graph too."""
    lm, V, rng = model
    ids = torch.from_numpy(np.random.default_rng(3).integers(0, V, (3, 40)).astype(np.int32)).cuda()
    want = lm.prefill(ids)
    st = lm.new_states(3)
    lm.prefill(ids[:, :38].contiguous(), st)
    lm.decode(ids[:, 38].contiguous(), st)
    saved = [tuple(t.clone() for t in pair) for pair in st]
    assert torch.equal(lm.decode(ids[:, 39].contiguous(), st), want)
    x, h = (torch.empty(3, 256, device="cuda") for _ in range(2))
    ws, bufs, last = lm.stack.layers[0].workspace(3, 1), lm.head_buffers(3), ids[:, 39].contiguous()
    for pair, old in zip(st, saved):
        for t, o in zip(pair, old):
            t.copy_(o)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = lm.decode(last, st, x, h, ws, bufs)
    graph.replay()
    torch.cuda.synchronize()
    lib.sync_status()
    assert torch.equal(y, want)
