"""The token loop's operators right behind the kernels they depend on, without a
synchronisation in between: the same bits as with one."""
import numpy as np
import pytest

from quantized_state_space_mamba2_b200 import synth as S

torch = pytest.importorskip("torch")
import token_plain as P  # noqa: E402

pytestmark = pytest.mark.gpu
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


def codes(N, K):
    return (torch.zeros(N, K, device="cuda", dtype=torch.int8).view(E4M3),
            torch.zeros(P.blocks(N), P.blocks(K), device="cuda"))


def test_prepared_weights_behind_their_writer_and_their_reader(lib):
    """A weight prepared from rows that the kernel before has just written, and
    into codes that the product before is still reading."""
    g = gen(1)
    V, K, N, M = 500, 2560, 4096, 2048
    table = randn(g, V, K)
    ids = [torch.randint(0, V, (N,), device="cuda", generator=g, dtype=torch.int32) for _ in range(4)]
    a, _ = codes(M, K)
    lib.prepare_linear_fp8(randn(g, M, K), a, torch.empty(M // 128, K // 128, device="cuda"))
    s_a = torch.exp(0.1 * randn(g, M, K // 128))

    def chain(sync):
        rows, (q, s) = torch.zeros(N, K, device="cuda"), codes(N, K)
        out = []
        torch.cuda.synchronize()
        for i in ids:
            y = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
            for call in (lambda: lib.embed_rows(i, table, rows),
                         lambda: lib.prepare_linear_fp8(rows, q, s),
                         lambda: lib.fp8_gemm(a, s_a, q, s, y)):
                call()
                if sync:
                    torch.cuda.synchronize()
            out.append(y)
        torch.cuda.synchronize()
        return out + [q.view(torch.uint8), s]

    want = chain(True)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(chain(False), want))
    lib.sync_status()


@pytest.mark.parametrize("bits", [31, 16])
def test_a_decode_step_right_behind_the_reordering_of_its_state(lib, bits):
    """fm_reorder_rows, then the scan of one token on the moved states; also with a
    decode-size GEMM between them, which lets its successor start before it waits
    itself."""
    s = S.MAMBA2_2P7B
    B, beams = 4, 8
    rows, cc, nh = B * beams, s.conv_ch, s.nheads
    g = gen(bits)
    ints = lambda lo, hi, *shape: torch.randint(lo, hi, shape, device="cuda", generator=g)
    xbc = ints(-127, 128, rows, 1, cc).to(torch.int8)
    dt_raw = randn(g, rows, 1, nh)
    X = lib.exp_table_layout(s)
    exps = np.zeros(X.size, np.int32)
    exps[X.e_x:X.e_x + nh], exps[X.e_B], exps[X.e_C] = -4, -4, -3
    exps[X.e_h:X.e_h + nh], exps[X.e_y:X.e_y + nh], exps[X.e_D:X.e_D + nh] = -18, -23, -10
    exps = torch.from_numpy(exps).cuda()
    dt_bias, A_q, D_q = randn(g, nh), ints(-4096, 0, nh).int(), ints(-999, 999, nh).int()
    parents = [ints(0, beams, B, beams).int() for _ in range(6)]
    a, w = ints(-127, 128, rows, 512).to(torch.int8), ints(-127, 128, 512, 512).to(torch.int8)
    one, y2 = torch.ones(512, device="cuda"), torch.empty(rows, 512, device="cuda")
    lib.set_state_spec(bits, 0 if bits == 31 else 7)
    try:
        dtype = torch.int32 if bits == 31 else torch.int16
        lim = 2 ** 26 if bits == 31 else 16000
        first = ints(-lim, lim, rows, nh, s.headdim, s.d_state).to(dtype)
        ws = torch.empty(max(lib.scan_workspace_bytes(s, rows, 1), 16), dtype=torch.uint8, device="cuda")

        def chain(sync, between):
            state = first.clone()
            kept, y = lib.RowSet([state]), torch.empty(rows, 1, s.d_inner, dtype=torch.int32, device="cuda")
            out = []
            torch.cuda.synchronize()
            for parent in parents:
                lib.reorder_rows(kept, parent)
                if sync:
                    torch.cuda.synchronize()
                if between:
                    lib.w8a8_gemm(a, one[:rows], w, one, y2)
                lib.ssm_scan_pot(xbc, dt_raw, rows, 1, s, dt_bias, A_q, D_q, exps, state, y, ws)
                if sync:
                    torch.cuda.synchronize()
                out.append(y.clone())
            torch.cuda.synchronize()
            return out + [state]

        want = chain(True, False)
        for between in (False, True):
            for _ in range(3):
                assert all(torch.equal(x, y) for x, y in zip(chain(False, between), want))
        lib.sync_status()
    finally:
        lib.set_state_spec(31, 0)
