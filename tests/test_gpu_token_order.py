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
