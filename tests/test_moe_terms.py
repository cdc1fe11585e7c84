"""What the experts' FP4 terms keep of an activation, format by format: calls whose result hangs on the
last digits, bit for bit, and the bound of each format on its own. The reference is plain arithmetic in
64 bits; the CPU tests show that it tells a split with any one term lost."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_14_b200 as nv
import test_moe as M

TERMS = 8
FORMATS = ["mxfp4", "nvfp4"]


def split(v, block, reach):
    """The terms of a row of values, [8, n], from their definition: with E the exponent of the largest
    of a block (at least the row's less `reach`), v / 2^(E - 21) rounded to an integer and written to
    base 8 with the digits -4 .. 3, the first digit at 2^E. E is at least -106."""
    v = np.asarray(v, np.float64)
    exponent = lambda b: np.frexp(np.abs(b).max())[1] - 1 if b.any() else -106  # noqa: E731
    least = max(exponent(v) - reach, -106)
    out = np.zeros((TERMS, v.size))
    for i in range(0, v.size, block):
        b = v[i:i + block]
        e = max(exponent(b), least)
        x = np.rint(b / 2.0 ** (e - 21)).astype(np.int64)
        for j in range(TERMS - 1, -1, -1):
            d = (x + 4) % 8 - 4
            x = (x - d) // 8
            out[j, i:i + block] = d * 2.0 ** (e - 3 * j)
        assert (x == 0).all()
    return out


def terms_of(v, fmt):
    return split(v, 32, 300) if fmt == "mxfp4" else split(v, 16, 17)


# ---- calls that hang on one digit -------------------------------------------------------------
#
# One expert, F = 64. Token j has 1.5 twice in the first block, met by weights +6 and -6 (their
# difference is exactly 0), and beside them 3 * 2^(-3 j), which the block's digit j alone holds. 2^15
# in a block of its own, met by no weight, makes the row's largest value that of another block. All
# sums are of few small integers times powers of two: exact in fp32, and every result in bf16.

H, F = 128, 64
PICK = np.array([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.5, -1.0, -3.0, -6.0])


def digit(j):
    return 3.0 * 2.0 ** (-3 * j) if j else 1.0  # (3 would be the block's largest)


def call_on_x(j):
    """x whose own block cancels down to digit j: x, gate_up [2F, H], down [H, F], y."""
    x = np.zeros(H)
    x[0] = x[1] = 1.5
    x[2] = digit(j)
    x[64], x[96] = 16.0, 2.0 ** 15
    up = np.zeros((2 * F, H))
    up[:F, 64] = 4.0                       # gate: 64, and silu(64) = 64
    up[F:, 0], up[F:, 1] = 6.0, -6.0
    w = PICK[np.arange(F) % PICK.size]
    up[F:, 2] = w
    down = np.zeros((H, F))
    down[np.arange(H), np.arange(H) % F] = 1.0
    return x, up, down, (64.0 * w * x[2])[np.arange(H) % F]


def call_on_h(j):
    """The same of h: values 0 and 1 of it are met by +6 and -6, value 2 is digit j of their block."""
    x = np.zeros(H)
    x[0] = 1.5
    x[32] = digit(j)
    x[64], x[96] = 16.0, 2.0 ** 15
    up = np.zeros((2 * F, H))
    up[:F, 64] = 4.0
    up[F, 0] = up[F + 1, 0] = up[F + 2, 32] = 1.0
    up[F + 48, 96] = 1.0                   # h's largest value, in another block
    down = np.zeros((H, F))
    w = PICK[np.arange(H) % PICK.size]
    down[:, 0], down[:, 1], down[:, 2] = 6.0, -6.0, w
    return x, up, down, 64.0 * w * x[32]


def compute(x, up, down, fmt, lose_x=None, lose_h=None):
    """y from the terms, one of x's or of h's left out."""
    def cut(v, lose):
        t = terms_of(v, fmt)
        if lose is not None:
            t[lose] = 0.0
        return t.sum(0)
    a = up @ cut(x, lose_x)
    with np.errstate(over="ignore"):
        h = a[:F] / (1.0 + np.exp(-a[:F])) * a[F:]
    return down @ cut(h, lose_h)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("j", range(TERMS))
def test_each_call_hangs_on_its_digit(fmt, j):
    for call, name in ((call_on_x, "lose_x"), (call_on_h, "lose_h")):
        x, up, down, y = call(j)
        assert torch.equal(torch.from_numpy(x).bfloat16().double(), torch.from_numpy(x))
        assert np.array_equal(torch.from_numpy(y).bfloat16().double().numpy(), y)
        assert np.array_equal(compute(x, up, down, fmt), y)
        assert not np.array_equal(compute(x, up, down, fmt, **{name: j}), y)


@pytest.mark.parametrize("fmt,block,reach", [("mxfp4", 32, 300), ("nvfp4", 16, 17)])
def test_split_keeps_the_bound(fmt, block, reach):
    g = np.random.default_rng(3)
    for _ in range(50):
        v = g.standard_normal(128) * np.exp2(g.integers(-30, 12, 128 // block).repeat(block))
        t = terms_of(v, fmt)
        err = np.abs(t.sum(0) - v)
        assert (err <= terms_error(torch.from_numpy(v), fmt).numpy()).all()


def as_experts(w, fmt):
    """One expert with the E2M1 values w and scales of 1."""
    mags = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    n = np.abs(np.abs(w)[..., None] - mags).argmin(-1)
    assert np.array_equal(mags[n], np.abs(w))
    n = n + 8 * (w < 0)
    codes = torch.from_numpy((n[:, 0::2] | n[:, 1::2] << 4).astype(np.uint8)).cuda()[None]
    b, one = (32, 127) if fmt == "mxfp4" else (16, 0x38)
    s = torch.full((1, w.shape[0], w.shape[1] // b), one, dtype=torch.uint8, device="cuda")
    return nv.ExpertWeights(codes.contiguous(), s,
                            None if fmt == "mxfp4" else torch.ones(1, device="cuda"))


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.load()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("call", [call_on_x, call_on_h])
def test_every_digit_reaches_y(cuda, fmt, call):
    calls = [call(j) for j in range(TERMS)]
    x = torch.from_numpy(np.stack([c[0] for c in calls])).bfloat16().cuda()
    up, down = as_experts(calls[0][1], fmt), as_experts(calls[0][2], fmt)
    ids = torch.zeros(TERMS, 1, dtype=torch.int32, device="cuda")
    y = nv.moe_experts(x, ids, torch.ones(TERMS, 1, device="cuda"), up, down)
    got, ref = y.double().cpu().numpy(), np.stack([c[3] for c in calls])
    assert np.array_equal(got, ref), [j for j in range(TERMS) if not np.array_equal(got[j], ref[j])]


# ---- the bound of each format -----------------------------------------------------------------


def terms_error(v, fmt):
    """What eight terms leave of v at most. MXFP4: 2^-22 of the largest of a block of 32. NVFP4: 2^-22 of
    the largest of a block of 16, or of 2^-17 of the row's largest where that is more. Both: 2^-128."""
    b = 32 if fmt == "mxfp4" else 16
    top = v.abs().view(-1, b).max(-1).values.repeat_interleave(b)
    if fmt == "nvfp4":
        top = top.clamp(min=2.0 ** -17 * float(v.abs().max()))
    return 2.0 ** -22 * top + 2.0 ** -128


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,F,E,k", [(1, 2048, 1408, 2, 1), (5, 96, 416, 4, 3), (17, 288, 224, 2, 1),
                                       (20, 1056, 1312, 2, 2), (64, 512, 256, 8, 8)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("spike", [1.0, 1280.0, 20480.0])
def test_experts_within_their_formats_bound(cuda, monkeypatch, T, H, F, E, k, fmt, spike):
    """A channel of x far above the others, on which the weights are a thousandth of theirs."""
    monkeypatch.setattr(M, "terms_error", lambda v: terms_error(v, fmt))
    def quant(w):
        if fmt == "mxfp4":
            q = nv.quantize_mxfp4(w, linear=True)
            return q, nv.dequantize_mxfp4(q).double()
        q = nv.quantize(w, linear=True)
        one = nv.NVFP4Tensor(q.codes, None, q.scales_lin, torch.ones(1, device="cuda"), *w.shape)
        return q, nv.dequantize(one).double() * q.global_scale.double()
    g = M.gen(T + F)
    ups, downs = [], []
    for _ in range(E):
        w = torch.randn(2 * F, H, device="cuda", generator=g) * 0.05
        w[:, :32] *= 1e-3
        ups.append(quant(w))
        downs.append(quant(torch.randn(H, F, device="cuda", generator=g) * 0.05))
    up, down = ((nv.stack_experts([q for q, _ in s]), torch.stack([v for _, v in s]))
                for s in (ups, downs))
    x = torch.randn(T, H, device="cuda", generator=g)
    x[:, 1] = spike
    ids, p = M.some_ids(T, k, E, 4)
    M.check_experts(x.bfloat16(), ids, p, up, down)


# ---- silu far below zero ----------------------------------------------------------------------
#
# Pairs of hidden values that almost cancel in y: h_a = silu(a) u_a and h_b = silu(b) u_b with gates
# near -72 and u_b taken to 16 bits such that h_b = h_a (1 + 2^-14). y = h_a - h_b shows errors of
# silu that are 2^-14 of what they are to y alone.

PAIRS, TOKENS = 16, 16


def silu_pairs(seed):
    """x [TOKENS, H] (all of bf16), gate_up, down, and with what of x: a, b, u_a, u_b, [TOKENS, PAIRS]."""
    g = np.random.default_rng(seed)
    bf = lambda v: torch.from_numpy(v).bfloat16().double().numpy()  # noqa: E731
    x = np.zeros((TOKENS, 128))
    x[:, :32] = 12.0 + g.integers(-2, 3, (TOKENS, 32)) / 16.0
    a, b = -6.0 * x[:, 0:32:2], -6.0 * x[:, 1:32:2]
    silu = lambda v: v / (1.0 + np.exp(-v))  # noqa: E731
    u_a = bf(np.exp2(20.0 + g.random((TOKENS, PAIRS))))
    u_b = silu(a) * u_a / silu(b) * (1.0 + 2.0 ** -14)
    hi = bf(u_b)
    lo = bf(u_b - hi)
    x[:, 32:48], x[:, 64:80], x[:, 96:112] = u_a, hi, lo
    up = np.zeros((64, 128))
    for q in range(PAIRS):
        up[2 * q, 2 * q] = up[2 * q + 1, 2 * q + 1] = -6.0
        up[32 + 2 * q, 32 + q] = up[33 + 2 * q, 64 + q] = up[33 + 2 * q, 96 + q] = 1.0
    down = np.zeros((128, 32))
    for q in range(PAIRS):
        down[q, 2 * q], down[q, 2 * q + 1] = 1.0, -1.0
    return x, up, down, (a, b, u_a, hi + lo)


def check_silu_pairs(y, parts, fmt):
    """y [TOKENS, PAIRS] against 64 bits. The products before silu are exact sums of few digits. Each
    hidden value: expf (1 unit in the last place, 2^-23), the sum, the division and the product with u
    (half of one each): 5 * 2^-24, and u itself, exact or rounded once: 2^-24. The terms leave 2^-22 of
    the block's largest of either value; the sum of two values' digits is exact in each column and the
    columns' sum is off by less than 2^-20 of y; y is rounded to bf16 once."""
    a, b, u_a, u_b = parts
    h = np.stack([a / (1.0 + np.exp(-a)) * u_a, b / (1.0 + np.exp(-b)) * u_b], -1)  # [T, q, 2]
    y_ref = h[..., 0] - h[..., 1]
    size = np.abs(h)
    block = size.reshape(TOKENS, -1, 16 if fmt == "nvfp4" else 32)
    top = block.max(-1, keepdims=True).repeat(block.shape[-1], -1).reshape(size.shape)
    err = (6 * 2.0 ** -24 * size + 2.0 ** -22 * top).sum(-1) + 2.0 ** -20 * np.abs(y_ref)
    tol = err + 2.0 ** -8 * (np.abs(y_ref) + err)
    return np.abs(y - y_ref) / tol


def single_silu(v, exp):
    e = exp(-v.astype(np.float32))
    return v.astype(np.float32) / (np.float32(1.0) + e)


@pytest.mark.parametrize("fmt", FORMATS)
def test_silu_check_tells_a_short_exponential(fmt):
    exact = lambda v: np.exp(v.astype(np.float64)).astype(np.float32)  # noqa: E731
    # exp as 2^(v log2 e) with the product rounded to fp32
    short = lambda v: np.exp2((v * np.float32(np.log2(np.e))).astype(np.float64)).astype(  # noqa: E731
        np.float32)
    x, up, down, parts = silu_pairs(1)
    assert torch.equal(torch.from_numpy(x).bfloat16().double(), torch.from_numpy(x))
    worst = {}
    for name, exp in (("exact", exact), ("short", short)):
        a, b, u_a, u_b = parts
        h = np.stack([single_silu(a, exp) * u_a.astype(np.float32),
                      single_silu(b, exp) * u_b.astype(np.float32)], -1).reshape(TOKENS, -1)
        h = np.stack([terms_of(r, fmt).sum(0) for r in h]).reshape(TOKENS, PAIRS, 2)
        y = torch.from_numpy(h[..., 0] - h[..., 1]).bfloat16().double().numpy()
        worst[name] = check_silu_pairs(y, parts, fmt).max()
    assert worst["exact"] <= 1.0 and worst["short"] > 1.5, worst


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seed", [1, 2])
def test_silu_far_below_zero(cuda, fmt, seed):
    x, up, down, parts = silu_pairs(seed)
    y = nv.moe_experts(torch.from_numpy(x).bfloat16().cuda(),
                       torch.zeros(TOKENS, 1, dtype=torch.int32, device="cuda"),
                       torch.ones(TOKENS, 1, device="cuda"), as_experts(up, fmt),
                       as_experts(down, fmt))
    y = y.double().cpu().numpy()
    assert (y[:, PAIRS:] == 0).all()
    off = check_silu_pairs(y[:, :PAIRS], parts, fmt)
    assert (off <= 1.0).all(), float(off.max())
