"""DeviceLM and the layers on a stream other than the current one."""
import numpy as np
import pytest

from quantized_state_space_mamba2_b200 import synth as S

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_state_space_mamba2_b200 import build, lib
    build.build()
    lib.load()
    return lib


def overwrite():
    """Allocate and fill, on the current stream, blocks of every size a call may
    have freed."""
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
            for k in range(9, 25) for n in [1 << k] * 6]
    return junk[-1]


def test_a_model_on_a_side_stream(lib):
    """prefill, decode and logits queued on a busy side stream, while the current
    stream allocates and fills: the bits of the calls on the current stream."""
    from quantized_state_space_mamba2_b200.model import DeviceLM
    shape = S.MixerShape(d_model=256, d_inner=512, headdim=64, d_state=128)
    V, rng = 301, np.random.default_rng(9)
    lm = DeviceLM([S.layer_params(shape, 80 + l) for l in range(3)], shape,
                  rng.normal(0, 0.3, (V, 256)).astype(np.float32), np.ones(256, np.float32), embed_scale=4.0)
    ids = torch.from_numpy(rng.integers(0, V, (2, 64)).astype(np.int32)).cuda()
    lm.calibrate(ids)
    more = ids[:, 0].contiguous()
    states = lm.new_states(2)
    want = [lm.prefill(ids, states), lm.decode(more, states), lm.logits(lm.embed(more))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 26, device="cuda")
    for _ in range(4):
        states2 = lm.new_states(2)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(40):
                busy.add_(1.0)
        got = [lm.prefill(ids, states2, stream=side)]
        overwrite()
        got.append(lm.decode(more, states2, stream=side))
        overwrite()
        got.append(lm.logits(lm.embed(more, stream=side), stream=side))
        overwrite()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for p, q in zip(states2, states) for a, b in zip(p, q))
    lib.sync_status()


def test_layers_on_a_side_stream(lib):
    """A layer and a stack prepared, calibrated and run on a busy side stream."""
    from quantized_state_space_mamba2_b200.model import DeviceLayer, DeviceStack
    shape = S.MixerShape(d_model=256, d_inner=512, headdim=64, d_state=128)
    params = [S.layer_params(shape, 90 + l) for l in range(2)]
    x = torch.from_numpy(S.activations(2, 40, 256, seed=3, n_outliers=4, outlier_scale=20.0,
                                       outlier_seed=4)).cuda()
    host, first = x.cpu().pin_memory(), x[:, 0].contiguous()

    def run(stream, between):
        out = []

        def keep(t):
            between()
            out.append(t)

        L = DeviceLayer(params[0], shape, prenorm=True, stream=stream)
        keep(L.calibrate(x, stream=stream))
        keep(L.prefill(x, stream=stream))
        states = L.new_states(2)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(20):
                busy.add_(1.0)
        keep(L.decode(first, *states, stream=stream))
        keep(L.lq_prefill(x, stream=stream))
        stack = DeviceStack(params, shape)
        stack.calibrate(x)
        rows = [x.clone() for _ in range(3)]
        back = torch.empty_like(host).pin_memory()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(20):
                busy.add_(1.0)
        keep(stack.prefill_(rows[0], stream=stream))
        keep(stack.prefill_pipelined_(rows[1], 2, stream=stream))
        keep(stack.prefill_host(host, back, rows[2], 2, stream=stream))
        torch.cuda.synchronize()
        return [t.cuda() for t in out] + list(states)

    busy = torch.zeros(1 << 26, device="cuda")
    want = run(None, lambda: None)
    side = torch.cuda.Stream()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(side, overwrite), want))
    lib.sync_status()
