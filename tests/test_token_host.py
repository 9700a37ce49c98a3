"""Host-side checks of the token loop's entry points that need no GPU: argument
validation before any launch, workspace sizes, and the plain 64-bit forms the
GPU tests compare against, each against its formula in another form."""
import ctypes as C
import math

import pytest

from quantized_state_space_mamba2_b200 import build as B

torch = pytest.importorskip("torch")
import token_plain as P  # noqa: E402

p = [C.c_void_p(0x100000 * (i + 1)) for i in range(12)]  # aligned, never dereferenced
odd = C.c_void_p(0x100004)
OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def so():
    B.build()
    from quantized_state_space_mamba2_b200 import lib
    return lib.load()


def test_status_name(so):
    assert so.fm_status_string(9) == b"FM_ERR_INDEX"


def norm(so, x=p[0], xt=0, ldx=256, res=p[1], ldr=256, M=4, K=256, w=p[2], eps=1e-5, qt=2, q=p[3],
         s=p[4], out=p[5], lds=256):
    return so.fm_add_norm_quant(x, xt, ldx, res, ldr, M, K, w, eps, qt, q, s, out, lds, None)


def test_norm_refusals(so):
    for bad in (dict(xt=2), dict(xt=3), dict(qt=0), dict(qt=1), dict(x=None), dict(w=None), dict(q=None),
                dict(s=None), dict(eps=-1.0), dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf)):
        assert norm(so, **bad) == ARG, bad
    for bad in (dict(K=0), dict(K=250), dict(K=16400, ldx=16400, ldr=16400, lds=16400), dict(M=-1),
                dict(M=1 << 31), dict(ldx=255), dict(ldx=258), dict(ldr=240), dict(lds=257)):
        assert norm(so, **bad) == SHAPE, bad
    for bad in (dict(x=odd), dict(res=odd), dict(w=odd), dict(q=odd), dict(s=odd), dict(out=odd)):
        assert norm(so, **bad) == ALIGN, bad
    assert norm(so, M=0, x=None) == OK


def test_prepare_and_product_refusals(so):
    assert so.fm_prepare_linear_fp8(None, 4, 32, p[0], p[1], None) == ARG
    assert so.fm_prepare_linear_fp8(p[0], 4, 40, p[1], p[2], None) == SHAPE
    assert so.fm_prepare_linear_fp8(p[0], 0, 32, p[1], p[2], None) == SHAPE
    assert so.fm_prepare_linear_fp8(odd, 4, 32, p[1], p[2], None) == ALIGN

    def gemm(A=p[0], sa=p[1], M=4, W=p[2], sw=p[3], N=100, K=256, Y=p[4], yt=0, ldy=100):
        return so.fm_fp8_gemm(A, sa, M, W, sw, N, K, Y, yt, ldy, None)

    for bad in (dict(A=None), dict(sa=None), dict(W=None), dict(sw=None), dict(Y=None), dict(yt=2),
                dict(yt=3), dict(yt=9)):
        assert gemm(**bad) == ARG, bad
    for bad in (dict(K=0), dict(K=-16), dict(K=100), dict(ldy=99), dict(M=-1), dict(N=-1), dict(M=1 << 40),
                dict(N=1 << 40, ldy=1 << 40)):
        assert gemm(**bad) == SHAPE, bad
    for bad in (dict(A=odd), dict(sa=odd), dict(W=odd), dict(sw=odd), dict(Y=odd)):
        assert gemm(**bad) == ALIGN, bad
    assert gemm(M=0, A=None) == OK and gemm(N=0, ldy=0, W=None) == OK


def test_embed_refusals(so):
    def emb(ids=p[0], M=4, t=p[1], tt=0, ts=None, V=100, K=256, x=p[2], ldx=256):
        return so.fm_embed_rows(ids, M, t, tt, ts, V, K, 1.0, x, ldx, None)

    for bad in (dict(ids=None), dict(t=None), dict(x=None), dict(tt=3), dict(tt=2)):  # e4m3 needs scales
        assert emb(**bad) == ARG, bad
    for bad in (dict(V=0), dict(V=1 << 31), dict(K=8), dict(K=0), dict(ldx=255), dict(ldx=257), dict(M=-1)):
        assert emb(**bad) == SHAPE, bad
    assert emb(x=odd) == ALIGN and emb(ids=odd) == ALIGN
    assert emb(M=0, ids=None) == OK


def test_beam_refusals_and_workspace(so):
    from quantized_state_space_mamba2_b200 import lib
    need = lib.beam_workspace_bytes(2, 4, 1000, 4)
    assert need > 0 and lib.beam_workspace_bytes(0, 4, 1000, 4) >= 0
    for bad in ((2, 33, 1000, 4), (2, 0, 1000, 4), (2, 4, 0, 4), (2, 4, 1 << 31, 4), (2, 4, 1000, 33),
                (2, 4, 1000, 0), (-1, 4, 1000, 4)):
        assert lib.beam_workspace_bytes(*bad) == 0, bad

    def sel(l=p[0], t=0, ld=1000, B=2, k=4, V=1000, sc=p[1], fin=None, eos=-1, n=4, o=p[2], par=p[3],
            tok=p[4], of=None, ws=p[5], nb=need):
        return so.fm_beam_select(l, t, ld, B, k, V, sc, fin, eos, n, o, par, tok, of, ws, nb, None)

    for bad in (dict(l=None), dict(t=2), dict(sc=None), dict(o=None), dict(par=None), dict(tok=None),
                dict(fin=p[6]), dict(eos=1000), dict(eos=-2), dict(o=p[1], n=3),
                dict(fin=p[6], of=p[6], eos=1, n=3)):
        assert sel(**bad) == ARG, bad
    for bad in (dict(k=33), dict(n=33), dict(n=0), dict(V=0), dict(ld=999), dict(B=-1)):
        assert sel(**bad) == SHAPE, bad
    for bad in (dict(l=odd), dict(sc=odd), dict(o=odd), dict(ws=odd)):
        assert sel(**bad) == ALIGN, bad
    assert sel(ws=None) == WS and sel(nb=need - 1) == WS
    assert sel(B=0, l=None) == OK


def test_reorder_refusals(so):
    def arr(*v):
        return (C.c_void_p * len(v))(*v)

    nb = (C.c_int64 * 2)(64, 128)

    def ro(src=arr(0x100000, 0x200000), dst=arr(0x100000, 0x200000), nbytes=nb, n=2, B=2, sb=4, db=4,
           par=p[9]):
        return so.fm_reorder_rows(src, dst, nbytes, n, B, sb, db, par, None)

    for bad in (dict(n=-1), dict(src=None), dict(dst=None), dict(nbytes=None), dict(par=None),
                dict(src=arr(0, 0x200000)), dict(sb=1),  # in place needs as many beams
                dict(src=arr(0x100000 + 16, 0x200000))):  # overlapping, not the same
        assert ro(**bad) == ARG, bad
    for bad in (dict(B=-1), dict(B=65536), dict(sb=33, db=33), dict(db=0), dict(nbytes=(C.c_int64 * 2)(64, -1))):
        assert ro(**bad) == SHAPE, bad
    assert ro(src=arr(0x100000, 0x200004), dst=arr(0x300000, 0x400000)) == ALIGN
    assert ro(n=0, src=None) == OK and ro(B=0) == OK


def test_python_checks(monkeypatch):
    """The binding refuses what the library could not see: types, shapes, strides
    and devices."""
    from quantized_state_space_mamba2_b200 import lib
    monkeypatch.setattr(lib, "_place", lambda stream: (-1, 0))  # host tensors stand for the device's
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    z, i8, i32, f8 = torch.zeros, torch.int8, torch.int32, torch.float8_e4m3fn
    whole = z(8, 4)
    lib.RowSet([whole[:4], whole[4:]])  # neighbours are no overlap
    lib.RowSet([z(4, 4), z(4, 4)], [whole[:4], whole[4:]])
    refused = [
        ("dtype", lambda: lib.add_norm_quant(z(2, 32, dtype=torch.float16), z(32), z(2, 32, dtype=i8), z(2))),
        ("shape", lambda: lib.add_norm_quant(z(2, 32), z(31), z(2, 32, dtype=i8), z(2))),
        ("shape", lambda: lib.add_norm_quant(z(2, 32), z(32), z(2, 32, dtype=i8), z(2, 1))),
        ("shape", lambda: lib.add_norm_quant(z(2, 32), z(32), z(2, 32).to(f8), z(2))),
        ("column stride", lambda: lib.add_norm_quant(z(32, 2).t(), z(32), z(2, 32, dtype=i8), z(2))),
        ("shape", lambda: lib.fp8_gemm(z(2, 32).to(f8), z(2, 1), z(3, 16).to(f8), z(1, 1), z(2, 3))),
        ("shape", lambda: lib.fp8_gemm(z(2, 32).to(f8), z(2, 1), z(3, 32).to(f8), z(1, 1), z(2, 4))),
        ("dtype", lambda: lib.fp8_gemm(z(2, 32), z(2, 1), z(3, 32).to(f8), z(1, 1), z(2, 3))),
        ("scales", lambda: lib.embed_rows(z(2, dtype=i32), z(4, 16), z(2, 16), table_s=z(1, 1))),
        ("scales", lambda: lib.embed_rows(z(2, dtype=i32), z(4, 16).to(f8), z(2, 16))),
        ("dtype", lambda: lib.embed_rows(z(2, dtype=torch.int64), z(4, 16), z(2, 16))),
        ("one stride", lambda: lib.beam_select(z(2, 5, 9)[:, :3], z(2, 3), z(2, 3), z(2, 3, dtype=i32),
                                               z(2, 3, dtype=i32), z(999))),
        ("dtype", lambda: lib.beam_select(z(2, 3, 9), z(2, 3), z(2, 3), z(2, 3, dtype=torch.int64),
                                          z(2, 3, dtype=i32), z(999))),
        ("rows", lambda: lib.reorder_rows(lib.RowSet([z(8, 4)]), z(2, 3, dtype=i32))),
        ("number of rows", lambda: lib.RowSet([z(8, 4), z(6, 4)])),
        ("shape", lambda: lib.RowSet([z(8, 4)], [z(2, 5)])),
        ("overlap", lambda: lib.RowSet([whole[:4], whole[2:6]])),
        ("overlap", lambda: lib.RowSet([whole[:4], whole[:4]])),
        ("overlap", lambda: lib.RowSet([z(4, 4), whole[:4]], [whole[2:6], z(4, 4)])),
    ]
    for i, (why, call) in enumerate(refused):
        with pytest.raises(ValueError, match=why):
            call()
            pytest.fail(f"refusal {i} ({why}) did not come")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(lib, "_place", lambda stream: (0, 0))
    with pytest.raises(ValueError, match="CUDA"):
        lib.add_norm_quant(z(2, 32), z(32), z(2, 32, dtype=i8), z(2))
    with pytest.raises(ValueError, match="CUDA"):
        lib.RowSet([z(8, 4)])


# ------------------------------------------------------------------ the plain forms
def test_plain_e4m3_is_the_types_rounding():
    v = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * torch.logspace(-4, 3, 20000)
    want = v.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert torch.equal(P.e4m3_round(v.double()).float(), want)


def test_plain_norm_and_product():
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(5, 400, generator=g), torch.ones(400)
    r, codes, s, sure = P.norm(x, x, w, 1e-5, "e4m3")
    assert torch.equal(r, x + x) and bool((sure == 1).all())
    y = torch.nn.functional.rms_norm((x + x).double(), (400,), eps=1e-5)
    assert float((P.dequant_rows(codes, s) - y).abs().max()) <= float(y.abs().max()) * 2.0 ** -4
    _, c8, s8, _ = P.norm(x, None, w, 1e-5, "int8")
    y = torch.nn.functional.rms_norm(x.double(), (400,), eps=1e-5)
    assert bool(((c8 * s8[:, None] - y).abs() <= 0.5001 * s8[:, None]).all())


def test_plain_beam_is_a_sort_of_all_candidates():
    g = torch.Generator().manual_seed(3)
    l, sc = torch.randn(3, 4, 50, generator=g) * 2, -torch.rand(3, 4, generator=g)
    out, par, tok, _ = P.beam(l, sc, None, -1, 7)
    c = torch.log_softmax(l.double(), 2) + sc.double()[:, :, None]
    v, i = torch.sort(c.view(3, -1), dim=1, descending=True, stable=True)
    assert torch.allclose(out, v[:, :7], rtol=0, atol=1e-12)
    assert torch.equal(par * 50 + tok, i[:, :7])


def test_a_model_on_a_side_stream_owns_its_buffers(monkeypatch):
    """stream= of DeviceLM: what a call allocates comes from that stream's memory
    and every step runs there (stand-ins for the kernels and the streams)."""
    import contextlib

    from quantized_state_space_mamba2_b200 import lib, model
    from quantized_state_space_mamba2_b200.synth import MixerShape
    now, made, ran = [None], [], []

    @contextlib.contextmanager
    def stream(s):
        old, now[0] = now[0], s if s is not None else now[0]
        yield
        now[0] = old

    def recorded(make):
        def f(*a, **kw):
            made.append(now[0])
            return make(*a, **kw)
        return f

    def step(name):
        def f(*a, stream=None, **kw):
            ran.append((name, now[0] if stream is None else stream))
        return f

    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    monkeypatch.setattr(lib, "add_norm_quant", step("norm"))
    monkeypatch.setattr(lib, "fp8_gemm", lambda *a: step("product")(stream=a[5] if len(a) > 5 else None))
    monkeypatch.setattr(lib, "embed_rows",
                        lambda *a: step("embed")(stream=a[5] if len(a) > 5 else None))
    shape = MixerShape(d_model=256, d_inner=512, headdim=64, d_state=128)

    class Layer:
        def workspace(self, B, T):
            return torch.empty(8)

        def prefill(self, x, stream=None, **kw):
            step("layer")(stream=stream)

        decode = lambda self, x, *states, stream=None, **kw: step("layer")(stream=stream)

    lm = object.__new__(model.DeviceLM)
    lm.shape, lm.embed_scale, lm.device = shape, 1.0, torch.device("cpu")
    lm.stack = type("Stack", (), {"layers": [Layer(), Layer()]})()
    lm.table, lm.table_s = lm.head, lm.head_s = torch.zeros(301, 256), torch.zeros(3, 2)
    lm.norm_w = torch.ones(256)
    ids, h = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(2, 256)
    calls = [lambda s: lm.embed(ids, stream=s), lambda s: lm.logits(h, stream=s),
             lambda s: lm.prefill(ids, stream=s),
             lambda s: lm.decode(ids[:, 0], [(None, None)] * 2, stream=s)]
    for want in ("side", None):
        for call in calls:
            made.clear()
            ran.clear()
            call(want)
            assert made and set(made) == {want}
            assert ran and {s for _, s in ran} == {want}
            assert now[0] is None


def test_a_layer_on_a_side_stream_owns_its_buffers(monkeypatch):
    """stream= of DeviceLayer and DeviceStack, with the same stand-ins."""
    import contextlib

    from quantized_state_space_mamba2_b200 import lib, model
    now, made, ran = [None], [], []

    @contextlib.contextmanager
    def stream(s):
        old, now[0] = now[0], s
        yield
        now[0] = old

    def recorded(make):
        def f(*a, **kw):
            made.append(now[0])
            return make(*a, **kw)
        return f

    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    for name in ("calib_workspace_bytes", "workspace_bytes", "lq_workspace_bytes", "stack_workspace_bytes"):
        monkeypatch.setattr(lib, name, lambda *a: 16)
    for name, last in (("calibrate_layer", 11), ("mixer_prefill", 9), ("decode_step", 8),
                       ("lq_mixer_prefill", 10), ("stack_prefill", 7), ("stack_prefill_host", 9)):
        monkeypatch.setattr(lib, name, lambda *a, last=last: ran.append(a[last] if len(a) > last else now[0]))
    L = object.__new__(model.DeviceLayer)
    L.__dict__.update(dict.fromkeys(("shape", "struct", "lq_struct", "conv_b", "exps", "conv_bq",
                                     "static_amax")), device=torch.device("cpu"))
    stack = object.__new__(model.DeviceStack)
    stack.shape, stack.layers = None, [L, L]
    x = torch.zeros(2, 5, 32)
    for call in (lambda: L.calibrate(x, stream="side"), lambda: L.prefill(x, stream="side"),
                 lambda: L.decode(x[:, 0], None, None, stream="side"), lambda: L.lq_prefill(x, stream="side"),
                 lambda: stack.prefill_(x, stream="side"), lambda: stack.prefill_pipelined_(x, stream="side"),
                 lambda: stack.prefill_host(x, x, x, stream="side")):
        made.clear()
        ran.clear()
        call()
        assert made and set(made) == {"side"} and ran and set(ran) == {"side"}
        assert now[0] is None


def test_beam_workspace_covers_smaller_selections(so):
    """A workspace sized for a selection serves every one of fewer sequences, beams,
    tokens or slots."""
    size = so.fm_beam_workspace_bytes
    for V in (1, 2048, 2049, 4096, 4097, 8193, 32001, 50000, 100003, 1 << 20, (1 << 31) - 1):
        for n in (1, 4, 8, 32):
            rows = [size(B, 1, V, n) for B in range(0, 320)]
            assert rows == sorted(rows), (V, n)
            for B in (1, 5, 12, 40):
                beams = [size(B, k, V, n) for k in range(1, 33)]
                assert beams == sorted(beams), (B, V, n)
            assert [size(7, 3, V, m) for m in range(1, 33)] == sorted(size(7, 3, V, m) for m in range(1, 33))
    for rows in (1, 3, 12, 40, 150, 300):
        by_v = [size(rows, 2, V, 4) for V in range(1, 200001, 511)]
        assert by_v == sorted(by_v), rows


def test_norm_refuses_sums_over_inputs_of_another_layout(so):
    """sum_out may be x or the residual only where each element lands on itself."""
    assert norm(so, xt=1, out=p[0]) == ARG                # bf16 x: the sums are twice as wide
    assert norm(so, ldx=264, out=p[0]) == ARG             # other row strides
    assert norm(so, out=p[0], lds=264) == ARG
    assert norm(so, ldr=260, out=p[1]) == ARG
    assert norm(so, M=0, xt=1, out=p[0]) == OK


def test_reorder_refuses_to_write_the_parents(so):
    def arr(*v):
        return (C.c_void_p * len(v))(*v)

    def ro(src, dst, nbytes, B=2, sb=4, db=4, par=0x900000):
        n = len(nbytes)
        return so.fm_reorder_rows(arr(*src), arr(*dst), (C.c_int64 * n)(*nbytes), n, B, sb, db, par, None)

    # the parents are read while the buffers are written: 2 x 4 of 4 bytes at 0x900000
    for at, rb in ((0x900000, 4), (0x900010, 4), (0x8FFFF0, 64), (0x8FF000, 0x300)):
        assert ro([at], [at], [rb]) == ARG, (at, rb)
        assert ro([0x100000, 0x200000], [0x100000, at], [64, rb]) == ARG, (at, rb)


def test_reorder_refuses_before_any_row_moves(so):
    """Rows too long for a launch are refused before another buffer's are moved."""
    def arr(*v):
        return (C.c_void_p * len(v))(*v)

    def ro(src, nbytes):
        n = len(nbytes)
        return so.fm_reorder_rows(arr(*src), arr(*src), (C.c_int64 * n)(*nbytes), n, 2, 4, 4, 1 << 50, None)

    long = (1 << 32) + 1  # bytes: no multiple of 4, moved one by one
    assert ro([0x100000], [long]) == SHAPE
    assert ro([1 << 44, 0x100000], [64, long]) == SHAPE
    assert ro([1 << 44, 0x100000], [64, 1 << 36]) == SHAPE


def test_row_set_of_any_iterable(monkeypatch):
    """A RowSet keeps the tensors of a generator for both sides."""
    from quantized_state_space_mamba2_b200 import lib
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # host tensors stand for the device's
    buffers = [torch.zeros(8, 4), torch.zeros(8, 3)]
    rows = lib.RowSet(t for t in buffers)
    assert all(a is b for side in (rows.dst, rows.src) for a, b in zip(side, buffers))
    assert len(rows.dst) == len(rows.src) == 2
    assert list(rows._dst) == list(rows._src) == [t.data_ptr() for t in buffers]
