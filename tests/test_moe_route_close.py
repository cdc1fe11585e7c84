"""The router where logits are equal or all but equal: the order is that of the exact logits, equal ones by
the lower expert, whatever the order and the rounding of a sum."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_14_b200 as nv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.load()


def rows_of_one_sum(E, H, seed, spread, signs=(-1, 1)):
    """[E, H] bf16 values: every row the same values, of `spread` binades, in an order of its own, and 64
    more columns of zeros. Their sums are multiples of 2^(-spread - 8) below 2^13: exact in fp64."""
    g = np.random.default_rng(seed)
    v = np.ldexp(1.0 + g.integers(0, 128, H) / 128.0, -g.integers(0, spread, H)) * g.choice(signs, H)
    w = np.stack([g.permutation(v) for _ in range(E)])
    return np.concatenate([w, np.zeros((E, 64))], 1), g


def bf16(v):
    t = torch.from_numpy(v).bfloat16()
    assert torch.equal(t.double(), torch.from_numpy(v))
    return t.cuda()


SIZES = [(1, 2048, 64, 4), (9, 960, 40, 8), (64, 4032, 128, 8), (3, 480, 512, 32), (300, 224, 16, 3),
         (5, 32, 2, 2)]


@pytest.mark.parametrize("T,H,E,k", SIZES)
@pytest.mark.parametrize("renorm", [True, False])
def test_equal_logits_by_the_lower_expert(T, H, E, k, renorm):
    w, g = rows_of_one_sum(E, H, T + E, 24)
    shut = E // 3
    bias = torch.zeros(E, device="cuda")
    bias[shut] = -np.inf
    scale = np.ldexp(1.0, g.integers(-3, 4, T))
    x = bf16(np.repeat(scale[:, None], H + 64, 1))
    for b, open_ in ((None, np.arange(E)), (bias, np.delete(np.arange(E), shut))):
        ids, p = nv.moe_route(x, bf16(w), k, bias=b, renormalize=renorm)
        n = min(k, open_.size)
        want = np.concatenate([open_[:n], np.full(k - n, -1)])
        assert (ids.cpu().numpy() == want).all()
        # equal logits: one over their number, within the division's and the sum's rounding
        share = 1.0 / (n if renorm else open_.size)
        assert (p[:, :n].double() - share).abs().max() <= 2.0 ** -20 * share
        assert (p[:, n:] == 0).all()


@pytest.mark.parametrize("T,H,E,k", SIZES)
@pytest.mark.parametrize("signs", [(-1, 1), (1, 1)])
def test_close_logits_in_their_exact_order(T, H, E, k, signs):
    """Logits that differ by multiples of 2^-24, through a column of their own, in a random order: far
    below the rounding of an fp32 sum of the others' sizes."""
    w, g = rows_of_one_sum(E, H, T + E + 1, 24, signs)
    rank = g.permutation(E)
    w[:, H + 1], w[:, H + 33] = rank % 16 / 16.0, 1.0 * (rank // 16)
    x = np.ones((T, H + 64))
    x[:, H:] = 2.0 ** -20
    ids, p = nv.moe_route(bf16(x), bf16(w), k)
    assert (ids.cpu().numpy() == np.argsort(-rank)[:k]).all()
    assert (p.double() - 1.0 / k).abs().max() <= 2.0 ** -12  # exp of up to 2^-15


def test_tokens_of_zeros():
    """A padded batch: the logits of a row of zeros are the bias, equal ones by the lower expert."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T, H, E, k = 30, 512, 96, 6
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    x[20:] = 0
    w = torch.randn(E, H, device="cuda", generator=g).bfloat16()
    ids, p = nv.moe_route(x, w, k)
    assert (ids[20:] == torch.arange(k, device="cuda")).all()
    assert ((p[20:].double() - 1 / k).abs() <= 2.0 ** -22).all()
    bias = torch.arange(E, device="cuda").float()
    assert (nv.moe_route(x, w, k, bias=bias)[0][20:] == torch.arange(E - 1, E - 1 - k, -1,
                                                                     device="cuda")).all()


def test_random_batches_in_the_order_of_64_bits():
    """Many tokens, experts and slots: pairs within 2^-24 of their sizes occur in each of these."""
    for seed, (T, H, E, k) in ((9, (2000, 672, 280, 31)), (61, (2000, 672, 280, 31)),
                               (34, (2000, 128, 310, 30)), (196, (2000, 5728, 212, 7))):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
        w = (torch.randn(E, H, device="cuda", generator=g) / H ** 0.5).bfloat16()
        z = x.double() @ w.double().T
        ref = torch.sort(z, dim=-1, descending=True, stable=True)[1][:, :k].int()
        ids = nv.moe_route(x, w, k)[0]
        # (where 64 bits themselves leave a pair open, either order)
        gap = (z.gather(1, ids.long()) - z.gather(1, ref.long())).abs()
        assert (gap <= 2.0 ** -49 * z.abs().max()).all()
