"""The experts kernel where a bounded wait gives up: no fault, the status word says NVFP4_ERR_TIMEOUT, the
call ends after about one limit, and the next call is right."""
import pytest
import torch

import nvfp4_block_scaled_14_b200 as nv
from nvfp4_block_scaled_14_b200 import _lib as L
from test_moe import gen, make_experts, some_ids

FAKE = 0x10000  # never dereferenced: each call below fails its host-side check first


def test_selftest_refusals():
    lib = L.load()
    n = lib.nvfp4_moe_workspace_bytes(4, 64, 64, 2)

    def call(T=4, absent=-1, wait=0, barrier=0):
        return lib.nvfp4_selftest_moe_experts(FAKE, T, 64, 64, 8, 2, FAKE, FAKE, 1, FAKE, FAKE, None,
                                              FAKE, FAKE, None, FAKE, FAKE, n, absent, wait, barrier,
                                              None)
    assert call(absent=-2) == L.NVFP4_ERR_INVALID_ARG
    assert call(wait=(1 << 20) + 1) == L.NVFP4_ERR_INVALID_ARG
    assert call(barrier=(1 << 21) + 1) == L.NVFP4_ERR_INVALID_ARG
    assert call(T=65) == L.NVFP4_ERR_SHAPE
    assert call(T=0) == L.NVFP4_OK


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.load()


T, H, F, E, K = 20, 512, 320, 4, 2


@pytest.fixture(scope="module", params=["mxfp4", "nvfp4"])
def layer(cuda, request):
    """(call with limits, reference y, y): one set of experts and tokens, y and its guard bytes."""
    fmt = request.param
    up, down = make_experts(E, 2 * F, H, fmt, 1)[0], make_experts(E, H, F, fmt, 2)[0]
    x = torch.randn(T, H, device="cuda", generator=gen(3)).bfloat16()
    ids, p = some_ids(T, K, E, 4)
    lib, pad = L.load(), 256
    n = lib.nvfp4_moe_workspace_bytes(T, H, F, K)
    ws = torch.zeros(n + 2 * pad, dtype=torch.uint8, device="cuda")
    y = torch.zeros(T * H * 2 + 2 * pad, dtype=torch.uint8, device="cuda")
    gs = lambda w: None if w.global_scale is None else w.global_scale.data_ptr()  # noqa: E731
    format_ = L.NVFP4_EXPERTS_MXFP4 if fmt == "mxfp4" else L.NVFP4_EXPERTS_NVFP4

    def call(absent=-1, wait=1 << 20, barrier=1 << 21):
        ws.fill_(0xA5)
        y.fill_(0xA5)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        st = lib.nvfp4_selftest_moe_experts(
            x.data_ptr(), T, H, F, E, K, ids.data_ptr(), p.data_ptr(), format_, up.codes.data_ptr(),
            up.scales.data_ptr(), gs(up), down.codes.data_ptr(), down.scales.data_ptr(), gs(down),
            y.data_ptr() + pad, ws.data_ptr() + pad, n, absent, wait, barrier,
            torch.cuda.current_stream().cuda_stream or None)
        end.record()
        assert st == L.NVFP4_OK
        status = nv.sync_status()
        for b in (ws, y):
            assert (b[:pad] == 0xA5).all() and (b[-pad:] == 0xA5).all()
        return status, y[pad:-pad].view(torch.bfloat16).view(T, H), start.elapsed_time(end)
    return call, nv.moe_experts(x, ids, p, up, down)


@pytest.mark.gpu
def test_full_limits_are_the_call(layer):
    call, ref = layer
    status, y, _ = call()
    assert status == 0 and torch.equal(y, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("limits", [dict(barrier=0), dict(wait=0), dict(wait=0, barrier=0),
                                    dict(absent=3, barrier=64), dict(absent=0, barrier=64)])
def test_given_up_call_is_reported_and_the_next_is_right(layer, limits):
    call, ref = layer
    for _ in range(2):
        status, _, _ = call(**limits)
        assert status == L.NVFP4_ERR_TIMEOUT
        assert nv.sync_status() == 0  # reported once
        status, y, _ = call()
        assert status == 0 and torch.equal(y, ref)


@pytest.mark.gpu
def test_only_the_first_barrier_is_waited_for(layer):
    """The call has three or four grid barriers. Against the time that one barrier takes to give up (the
    grid exchange's self-test, the same poll loop with as many CTAs): less than two of them."""
    call, ref = layer
    lib, limit = L.load(), 1 << 16
    n = torch.cuda.get_device_properties(0).multi_processor_count
    vals, out = torch.ones(n, device="cuda"), torch.zeros(2, device="cuda")
    ws = torch.zeros(lib.nvfp4_workspace_bytes(L.NVFP4_OP_QUANTIZE, 1, 0, 32), dtype=torch.uint8,
                     device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    assert lib.nvfp4_selftest_grid_exchange(n, vals.data_ptr(), 5, -1, 0, limit, out.data_ptr(),
                                            ws.data_ptr(), ws.numel(),
                                            torch.cuda.current_stream().cuda_stream or None) == 0
    end.record()
    assert nv.sync_status() == L.NVFP4_ERR_TIMEOUT
    one = start.elapsed_time(end)
    status, _, ms = call(absent=5, barrier=limit)
    assert status == L.NVFP4_ERR_TIMEOUT
    assert ms < 2 * one + 3.0, (ms, one)  # 1 ms for copies in flight, and the call itself
    status, y, _ = call()
    assert status == 0 and torch.equal(y, ref)


@pytest.mark.gpu
def test_binding_types(cuda):
    up, down = make_experts(2, 128, 64, "mxfp4", 1)[0], make_experts(2, 64, 64, "mxfp4", 2)[0]
    x = torch.zeros(2, 64, device="cuda", dtype=torch.bfloat16)
    ids, p = some_ids(2, 2, 2, 1)
    for bad in (lambda: nv.moe_experts(x, ids.tolist(), p, up, down),
                lambda: nv.moe_experts(x, None, p, up, down),
                lambda: nv.moe_experts(x, ids, p, nv.ExpertWeights(None, up.scales), down)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: nv.moe_experts(x, ids, None, up, down),
                lambda: nv.moe_experts(x, ids, p, nv.ExpertWeights(up.codes, None), down),
                lambda: nv.moe_experts(x, ids, p, up, nv.ExpertWeights(None, down.scales))):
        with pytest.raises(ValueError):
            bad()
    q = nv.quantize_mxfp4(x)
    for bad in (lambda: nv.linear_mxfp4(nv.MXFP4Tensor(None, q.scales_swz, None, 2, 64), q),
                lambda: nv.dequantize_mxfp4(nv.MXFP4Tensor(None, None, None, 2, 64))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        nv.linear_mxfp4(q, nv.MXFP4Tensor(None, q.scales_swz, None, 2, 64))
