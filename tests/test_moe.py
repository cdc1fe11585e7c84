"""Mixture-of-experts router and experts: refusals on the host, ids exactly and weights, outputs
within derived bounds of the 64-bit definition (plain torch in float64)."""
import math

import pytest
import torch

import nvfp4_block_scaled_14_b200 as nv
from nvfp4_block_scaled_14_b200 import _lib as L

FAKE = 0x10000  # never dereferenced: each call below fails its host-side check first


@pytest.fixture(scope="module")
def lib():
    return L.load()


# ---- refusals (no GPU) -----------------------------------------------------------------------


def test_route_refusals(lib):
    r = lib.nvfp4_moe_route
    call = lambda T=4, H=64, E=8, k=2, x=FAKE, w=FAKE, b=None, ids=FAKE, p=FAKE: \
        r(x, w, b, T, H, E, k, 1, ids, p, None)  # noqa: E731
    assert call(T=-1) == L.NVFP4_ERR_SHAPE
    assert call(H=40) == L.NVFP4_ERR_SHAPE
    assert call(E=0, k=1) == L.NVFP4_ERR_SHAPE
    assert call(E=513) == L.NVFP4_ERR_SHAPE
    assert call(k=0) == L.NVFP4_ERR_SHAPE
    assert call(k=9) == L.NVFP4_ERR_SHAPE
    assert call(E=64, k=33) == L.NVFP4_ERR_SHAPE
    assert call(x=None) == L.NVFP4_ERR_INVALID_ARG
    assert call(ids=None) == L.NVFP4_ERR_INVALID_ARG
    assert call(w=FAKE + 8) == L.NVFP4_ERR_ALIGNMENT
    assert call(b=FAKE + 2) == L.NVFP4_ERR_ALIGNMENT
    assert call(T=0, x=None, w=None, ids=None, p=None) == L.NVFP4_OK


def test_experts_refusals(lib):
    f = lib.nvfp4_moe_experts
    ws = lib.nvfp4_moe_workspace_bytes(4, 64, 64, 2)
    assert ws >= 4 * 2 * 64 * 2
    assert lib.nvfp4_moe_workspace_bytes(65, 64, 64, 2) == 0

    def call(x=FAKE, T=4, H=64, F=64, E=8, k=2, ids=FAKE, p=FAKE, fmt=1, up=FAKE, ugs=None,
             down=FAKE, dgs=None, y=FAKE, wsp=FAKE, n=ws):
        return f(x, T, H, F, E, k, ids, p, fmt, up, FAKE, ugs, down, FAKE, dgs, y, wsp, n, None)
    assert call(fmt=2) == L.NVFP4_ERR_INVALID_ARG
    assert call(T=65) == L.NVFP4_ERR_SHAPE
    assert call(T=-1) == L.NVFP4_ERR_SHAPE
    assert call(H=48) == L.NVFP4_ERR_SHAPE
    assert call(F=0) == L.NVFP4_ERR_SHAPE
    assert call(E=513) == L.NVFP4_ERR_SHAPE
    assert call(k=33) == L.NVFP4_ERR_SHAPE
    assert call(E=512, F=1 << 21) == L.NVFP4_ERR_SHAPE       # 2^31 stacked gate/up rows
    assert call(E=512, H=1 << 22) == L.NVFP4_ERR_SHAPE       # 2^31 stacked down rows
    assert call(x=None) == L.NVFP4_ERR_INVALID_ARG
    assert call(fmt=0) == L.NVFP4_ERR_INVALID_ARG            # NVFP4 without global scales
    assert call(fmt=0, ugs=FAKE, dgs=FAKE + 2) == L.NVFP4_ERR_ALIGNMENT
    assert call(up=FAKE + 8) == L.NVFP4_ERR_ALIGNMENT
    assert call(ids=FAKE + 2) == L.NVFP4_ERR_ALIGNMENT
    assert call(n=ws - 1) == L.NVFP4_ERR_WORKSPACE
    assert call(wsp=None) == L.NVFP4_ERR_WORKSPACE
    assert call(T=0, x=None, y=None) == L.NVFP4_OK


def test_binding_refusals():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    e = nv.ExpertWeights(torch.zeros(2, 64, 32, dtype=torch.uint8),
                         torch.zeros(2, 64, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        nv.moe_route(x, x, 1)
    with pytest.raises(TypeError):
        nv.moe_experts(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), e, e)
    with pytest.raises(TypeError):
        nv.stack_experts([])
    with pytest.raises(ValueError):
        nv.stack_experts([nv.MXFP4Tensor(x, x, None, 2, 64)])


# ---- router (GPU) ----------------------------------------------------------------------------


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def route_reference(x, w, k, bias, renorm):
    z = x.double() @ w.double().T
    if bias is not None:
        z = z + bias.double()
    z = torch.where(z.isnan(), -math.inf, z)
    s, ids = torch.sort(z, dim=-1, descending=True, stable=True)
    s, ids = s[:, :k], ids[:, :k]
    top = s[:, :1]
    ex = lambda v: torch.where(v == top, 1.0, torch.exp(v - top)).nan_to_num(0.0)  # noqa: E731
    p = torch.where(s > -math.inf, ex(s), 0.0)
    n = p.sum(-1, keepdim=True) if renorm else \
        torch.where(z > -math.inf, ex(z), 0.0).sum(-1, keepdim=True)
    p = torch.where(s > -math.inf, p / n.clamp(min=1e-300), 0.0)
    return torch.where(s > -math.inf, ids, -1).int(), p


def check_route(x, w, k, bias=None, renorm=True):
    ids, p = nv.moe_route(x, w, k, bias=bias, renormalize=renorm)
    ref_ids, ref = route_reference(x, w, k, bias, renorm)
    assert ids.dtype == torch.int32 and p.dtype == torch.float32
    assert torch.equal(ids, ref_ids)
    # A logit is off by its 32-term fp32 sums, two MMAs each off by at most two units in the last
    # place (2^-22) of its terms' sizes, 8 * 2^-24 of the sum of the products' sizes (S) in all,
    # and by the rounding of z - max to fp32 (2^-24 of at most 2 S'); an exponential turns an
    # absolute error d into a relative one of d, twice (numerator and denominator); expf and the
    # division add 2^-22, the sum of up to 512 terms 2^-24 a term in the worst order.
    S = (x.double().abs() @ w.double().abs().T).max() + (0.0 if bias is None else
                                                         bias[bias.isfinite()].abs().max())
    tol = float(2 * (8 + 2) * 2.0 ** -24 * S + 2.0 ** -20)
    assert ((p.double() - ref).abs() <= tol * ref.abs() + 2.0 ** -126).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E,k", [(1, 64, 4, 1), (1, 4096, 64, 4), (3, 2080, 40, 8),
                                     (16, 1024, 1, 1), (17, 96, 130, 32), (33, 512, 512, 8),
                                     (64, 4096, 128, 8), (301, 256, 96, 6)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(cuda, T, H, E, k, renorm):
    g = gen(T + E)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    w = (torch.randn(E, H, device="cuda", generator=g) / H ** 0.5).bfloat16()
    bias = torch.randn(E, device="cuda", generator=g)
    check_route(x, w, k, None, renorm)
    check_route(x, w, k, bias, renorm)


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masks_ties_and_nonfinite(cuda, renorm):
    g = gen(1)
    T, H, E, k = 6, 64, 12, 4
    # small integers: exact logits, many ties
    x = torch.randint(-1, 2, (T, H), device="cuda", generator=g).bfloat16()
    w = torch.randint(-1, 2, (E, H), device="cuda", generator=g).bfloat16()
    w[5:9] = w[4]
    check_route(x, w, k, None, renorm)
    bias = torch.zeros(E, device="cuda")
    for open_ in (0, 1, 3, 4, 12):
        bias[:] = -math.inf
        bias[torch.randperm(E, device="cuda", generator=g)[:open_]] = 0.5
        if open_:
            check_route(x, w, k, bias, renorm)
        ids, p = nv.moe_route(x, w, k, bias=bias, renormalize=renorm)
        assert ((ids >= 0).sum(1) == min(open_, k)).all()
        assert (p[ids < 0] == 0).all() and p.isfinite().all()
    # a NaN logit is never chosen, and spoils no other token
    y = x.clone()
    y[2, 3] = float("nan")
    ids, p = nv.moe_route(y, w, k)
    assert (ids[2] == -1).all() and (p[2] == 0).all()
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(ids[keep], nv.moe_route(x, w, k)[0][keep])
    bias = torch.zeros(E, device="cuda")
    bias[7] = math.inf
    ids, p = nv.moe_route(x, w, k, bias=bias, renormalize=renorm)
    assert (ids[:, 0] == 7).all() and (p[:, 0] == 1).all() and (p[:, 1:] == 0).all()


@pytest.mark.gpu
def test_route_checks(cuda):
    x = torch.zeros(2, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: nv.moe_route(x, w, 9), lambda: nv.moe_route(x, w, 0),
                lambda: nv.moe_route(x, w[:, :32], 2),
                lambda: nv.moe_route(x, w, 2, bias=torch.zeros(7, device="cuda")),
                lambda: nv.moe_route(x, w.cpu(), 2)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        nv.moe_route(x, w, 2, bias=torch.zeros(8, device="cuda", dtype=torch.float64))
    ids, p = nv.moe_route(x[:0], w, 2)
    assert ids.shape == (0, 2) and p.shape == (0, 2)


# ---- experts (GPU) ---------------------------------------------------------------------------


def make_experts(E, rows, cols, fmt, seed, std=0.05):
    g = gen(seed)
    ws = [torch.randn(rows, cols, device="cuda", generator=g) * std for _ in range(E)]
    if fmt == "mxfp4":
        q = [nv.quantize_mxfp4(w, linear=True) for w in ws]
        vals = [nv.dequantize_mxfp4(v).double() for v in q]
    else:
        q = [nv.quantize(w, linear=True) for w in ws]
        vals = []
        for v in q:  # exact values: codes x E4M3 x global scale
            one = nv.NVFP4Tensor(v.codes, None, v.scales_lin, torch.ones(1, device="cuda"), rows,
                                 cols)
            vals.append(nv.dequantize(one).double() * v.global_scale.double())
    return nv.stack_experts(q), torch.stack(vals)


def blocks_max(v):
    """Largest magnitude of each value's 32-block."""
    return v.abs().view(-1, 32).max(-1).values.repeat_interleave(32)


def terms_error(v):
    """Bound on what eight FP4 terms leave of v: half a unit of a fixed-point number. MXFP4: of units
    2^-21 of the power of two at or below the block's largest value. NVFP4: units of 2^-9, the row's
    largest value being divided to 2^8 or more: 2^-18 of it."""
    return 2.0 ** -22 * blocks_max(v) + 2.0 ** -18 * v.abs().max()


def experts_reference(x, ids, p, up, down):
    """y and a bound on |y_kernel - y| before y's own rounding, in float64.

    a = Wg x: inputs off by terms_error, and fp32 sums over the terms, whose sizes add up to at most
    4 |x| a value (digits of -4 .. 3 to base 8: with a leading digit d >= 1 in size the ones behind
    add up to at most 4/7 of its unit, so |x| >= 3/7 and the sizes are at most d + 4/7; the ratio is
    largest at d = 1, 11/3): K/16 additions, each off by at most 2^-22 of the sum of the sizes. silu has
    slope at most 1.1 and |silu(a)| <= |a|; expf, the division and the products add 2^-20 relative.
    h is kept in fp32 and enters the down product the same way; the weighted sum over rows and
    splits adds 2^-18 relative of its terms' sizes."""
    T, H = x.shape
    F = down.shape[2]
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(y)
    x = x.double()

    def product_error(w, v, dv):
        w = w.abs()
        sizes = w @ (4 * (v.abs() + dv))
        return w @ (dv + terms_error(v.abs() + dv)) + v.numel() / 16 * 2.0 ** -22 * sizes
    for t in range(T):
        for s in range(ids.shape[1]):
            e = int(ids[t, s])
            if not 0 <= e < up.shape[0]:
                continue
            a, da = up[e] @ x[t], product_error(up[e], x[t], torch.zeros_like(x[t]))
            gate, upv = a[:F], a[F:]
            act = gate / (1 + torch.exp(-gate))
            h = act * upv
            dh = (1.1 * da[:F] + 2.0 ** -20 * act.abs()) * (upv.abs() + da[F:]) \
                + act.abs() * da[F:]
            w = float(p[t, s])
            y[t] += w * (down[e] @ h)
            size = down[e].abs() @ (h.abs() + dh)
            err[t] += abs(w) * (product_error(down[e], h, dh) + 2.0 ** -18 * size)
    return y, err


def check_experts(x, ids, p, up, down):
    y = nv.moe_experts(x, ids, p, up[0], down[0])
    ref, err = experts_reference(x, ids, p, up[1], down[1])
    tol = err + 2.0 ** -8 * (ref.abs() + err)  # bf16: half a step
    off = (y.double() - ref).abs()
    assert y.dtype == torch.bfloat16 and y.shape == x.shape
    assert (off <= tol).all(), (float((off / tol.clamp(min=1e-300)).max()),
                                (off > tol).nonzero()[:4].tolist())
    return y


def some_ids(T, k, E, seed):
    g = gen(seed)
    ids = torch.stack([torch.randperm(E, device="cuda", generator=g)[:k] for _ in range(T)]).int()
    return ids, torch.rand(T, k, device="cuda", generator=g)


EXPERT_SHAPES = [(1, 32, 32, 1, 1), (1, 2048, 1408, 8, 4), (2, 160, 96, 3, 2), (5, 96, 416, 4, 3),
                 (8, 256, 256, 2, 2), (9, 128, 160, 1, 1), (17, 288, 224, 2, 1),
                 (33, 544, 64, 5, 4), (64, 512, 256, 8, 8), (64, 128, 128, 512, 2),
                 (64, 64, 32, 40, 32),      # the most rows
                 (16, 1056, 1312, 2, 2),    # scale rows that end inside a k-tile
                 (2, 9600, 64, 2, 2),       # one CTA per block of y
                 (5, 20480, 96, 3, 2)]      # more blocks of y than SMs


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,F,E,k", EXPERT_SHAPES)
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_experts(cuda, T, H, F, E, k, fmt):
    up, down = make_experts(E, 2 * F, H, fmt, 1), make_experts(E, H, F, fmt, 2)
    x = torch.randn(T, H, device="cuda", generator=gen(3)).bfloat16()
    x[:, 1] *= 300.0  # an outlier channel
    ids, p = some_ids(T, k, E, 4)
    y = check_experts(x, ids, p, up, down)
    assert torch.equal(y, nv.moe_experts(x, ids, p, up[0], down[0]))  # same bits again


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_experts_ids_outside_and_repeated(cuda, fmt):
    T, H, F, E, k = 7, 192, 96, 4, 5
    up, down = make_experts(E, 2 * F, H, fmt, 1), make_experts(E, H, F, fmt, 2)
    x = torch.randn(T, H, device="cuda", generator=gen(3)).bfloat16()
    ids, p = some_ids(T, 4, E, 4)
    ids = torch.cat([ids, ids[:, :1]], 1).contiguous()          # one expert twice
    p = torch.rand(T, k, device="cuda", generator=gen(5))
    ids[1] = -1                                                 # a token without experts
    ids[2] = torch.tensor([-1, 4, 2, 1 << 30, -(1 << 31)], dtype=torch.int32)
    ids[3] = 3                                                  # the same expert k times
    y = check_experts(x, ids, p, up, down)
    assert (y[1] == 0).all()
    none = torch.full_like(ids, -1)
    assert (nv.moe_experts(x, none, p, up[0], down[0]) == 0).all()
    # a weight that belongs to no expert is not read into the sum, whatever it is
    q = p.clone()
    q[1] = float("nan")
    q[2, [0, 1, 3, 4]] = float("inf")
    assert torch.equal(nv.moe_experts(x, ids, q, up[0], down[0]), y)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_experts_nonfinite_token_stays_alone(cuda, fmt):
    T, H, F, E, k = 10, 128, 64, 2, 2
    up, down = make_experts(E, 2 * F, H, fmt, 1), make_experts(E, H, F, fmt, 2)
    x = torch.randn(T, H, device="cuda", generator=gen(3)).bfloat16()
    ids, p = some_ids(T, k, E, 4)
    y = check_experts(x, ids, p, up, down)
    z = x.clone()
    z[4, 7] = float("nan")
    z[9, 100] = float("inf")
    out = nv.moe_experts(z, ids, p, up[0], down[0])
    keep = [i for i in range(T) if i not in (4, 9)]
    assert torch.equal(out[keep], y[keep])
    assert out[4].isnan().all() and (~out[9].isfinite()).all()
    # tiny and huge activations: the block exponents carry them
    for s in (2.0 ** -40, 2.0 ** 30):
        check_experts((x.double() * s).bfloat16(), ids, p, up, down)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_layer_quantize_route_experts(cuda, fmt):
    """Router and experts as a layer calls them, on weights quantized by the library's calls."""
    T, H, F, E, k = 12, 320, 160, 10, 3
    up, down = make_experts(E, 2 * F, H, fmt, 1), make_experts(E, H, F, fmt, 2)
    x = torch.randn(T, H, device="cuda", generator=gen(6)).bfloat16()
    w = (torch.randn(E, H, device="cuda", generator=gen(7)) / H ** 0.5).bfloat16()
    bias = torch.zeros(E, device="cuda")
    bias[3] = -math.inf
    ids, p = nv.moe_route(x, w, k, bias=bias)
    assert torch.equal(ids, route_reference(x, w, k, bias, True)[0]) and not (ids == 3).any()
    check_experts(x, ids, p, up, down)
    xs = torch.randn(2 * H, 2 * T, device="cuda", generator=gen(8)).bfloat16().T[::2, ::2]
    check_experts(xs, ids, p, up, down)  # strided activations


@pytest.mark.gpu
def test_experts_checks(cuda):
    up, down = make_experts(2, 128, 64, "mxfp4", 1), make_experts(2, 64, 64, "mxfp4", 2)
    nup, _ = make_experts(2, 128, 64, "nvfp4", 1)
    x = torch.zeros(2, 64, device="cuda", dtype=torch.bfloat16)
    ids, p = some_ids(2, 2, 2, 1)
    bad = [lambda: nv.moe_experts(x.repeat(33, 1), ids, p, up[0], down[0]),
           lambda: nv.moe_experts(x, ids, p, nup, down[0]),
           lambda: nv.moe_experts(x, ids[:1], p, up[0], down[0]),
           lambda: nv.moe_experts(x, ids, p, down[0], down[0]),
           lambda: nv.moe_experts(x, ids, p, up[0], up[0]),
           lambda: nv.moe_experts(x, ids, p, up[0], down[0],
                                  out=torch.empty(2, 65, device="cuda", dtype=torch.bfloat16)),
           lambda: nv.moe_experts(x, ids.cpu(), p, up[0], down[0])]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        nv.moe_experts(x, ids.long(), p, up[0], down[0])
    assert nv.moe_experts(x[:0], ids[:0], p[:0], up[0], down[0]).shape == (0, 64)


@pytest.mark.gpu
def test_experts_beside_guard_bytes(cuda):
    """y and the workspace lie between guard bytes; T odd, H and F that end inside a k-tile."""
    T, H, F, E, k = 5, 160, 96, 3, 2
    up, down = make_experts(E, 2 * F, H, "mxfp4", 1)[0], make_experts(E, H, F, "mxfp4", 2)[0]
    x = torch.randn(T, H, device="cuda", generator=gen(3)).bfloat16()
    ids, p = some_ids(T, k, E, 4)
    lib, pad = nv.load(), 256
    n = lib.nvfp4_moe_workspace_bytes(T, H, F, k)
    ws = torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    y = torch.full((T * H * 2 + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    st = lib.nvfp4_moe_experts(x.data_ptr(), T, H, F, E, k, ids.data_ptr(), p.data_ptr(), 1,
                               up.codes.data_ptr(), up.scales.data_ptr(), None,
                               down.codes.data_ptr(), down.scales.data_ptr(), None,
                               y.data_ptr() + pad, ws.data_ptr() + pad, n,
                               torch.cuda.current_stream().cuda_stream or None)
    assert st == 0
    torch.cuda.synchronize()
    for b in (ws, y):
        assert (b[:pad] == 0xA5).all() and (b[-pad:] == 0xA5).all()
    assert torch.equal(y[pad:-pad].view(torch.bfloat16).view(T, H),
                       nv.moe_experts(x, ids, p, up, down))


@pytest.mark.gpu
@pytest.mark.parametrize("T,fmt", [(1, "mxfp4"), (20, "nvfp4")])
def test_layer_captured_twice_and_replayed_together(cuda, T, fmt):
    """Two graphs of the layer, captured over one stream, replayed on two streams at once with new
    inputs, and both at once with eager calls: equal to the eager results, bit for bit."""
    H, F, E, k = 512, 256, 16, 4
    up, down = make_experts(E, 2 * F, H, fmt, 1)[0], make_experts(E, H, F, fmt, 2)[0]
    w = (torch.randn(E, H, device="cuda", generator=gen(7)) / H ** 0.5).bfloat16()
    xs = [torch.randn(T, H, device="cuda", generator=gen(10 + i)).bfloat16() for i in range(6)]
    layer = lambda x: nv.moe_experts(x, *nv.moe_route(x, w, k), up, down)  # noqa: E731
    eager = [layer(x) for x in xs]
    side, graphs = torch.cuda.Stream(), []
    for _ in range(2):
        inp = torch.empty_like(xs[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = layer(inp)
        graphs.append((g, inp, out))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(0, 6, 3):
        torch.cuda.synchronize()
        for s, (g, inp, _), x in zip(streams, graphs, xs[i:]):
            with torch.cuda.stream(s):
                inp.copy_(x)
                g.replay()
        with torch.cuda.stream(streams[2]):
            third = layer(xs[i + 2])
        torch.cuda.synchronize()
        for (_, _, out), ref in zip(graphs, eager[i:]):
            assert torch.equal(out, ref)
        assert torch.equal(third, eager[i + 2])
