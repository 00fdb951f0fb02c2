"""Attention over pages whose scales lie at the ends of their range, in both kernels (few rows, many rows),
against the 64-bit formulas.

Bounds: those of test_cache_gpu.py with the weight's rounding that the kernel in question has (fp16 2^-11 in the
few-rows kernel, bf16 2^-8 in the other), and half a step of bf16's subnormals, 2^-134.  In the few-rows kernel a query value is
off by up to 2^-22 of its row's largest; the queries here are of like size, so e_s covers it.  Its weights are fp16
numbers in units of 2^-15 of the row's largest P 2^exponent ("top"): below 2^-14 of the unit they are
multiples of 2^-24 of it, off by up to half of that, 2^-25 2^-15 = 2^-40 top, and a code is at most 448: n 448 2^-40 top
for n tokens.  (Beside ordinary values, 2^-31 of them; it counts where pages' scales are far apart.)
In the many-rows kernel keys and values of 2^128 and more count as bf16's largest, 255 * 2^120: a code 256
at exponent 120 is the only one that append writes, and the formulas get 255 in its place."""
import numpy as np
import pytest
import torch

from tests import cache_ref as ref
from tests.test_cache_gpu import bf16, i32, random_pool

pytestmark = pytest.mark.gpu

FEW, MANY = [1, 5], [70, 150]
CODE_256 = 0x78


def plain_of(pages):
    return [(ref.VALUES[c.cpu().numpy()], e.cpu().numpy()) for c, e in ((pages.k_codes, pages.k_exp), (pages.v_codes, pages.v_exp))]


def run(Q, pages, table, lens, causal=True):
    import top_routed_block_b200 as fv
    O, LSE, st = fv.fvattn_cache_attend(Q, pages, i32(table), i32(lens), causal=causal)
    fv.check_status(st, "attend")
    return O, LSE


def check(Q, got, plain, table, lens, causal=True, few=True):
    O, LSE = (x.double().cpu().numpy() for x in got)
    B, _, M, d = Q.shape
    o, lse, A, S = ref.attend(Q.double().cpu().numpy(), *plain[0], *plain[1], np.array(table), lens, [M] * B, causal)
    es = (d + 16) * 2.0 ** -24 * S
    n = max(lens)
    w = (2.0 ** -11 if few else 2.0 ** -8) + 2 * es + 2.0 ** -20 + n * 2.0 ** -24
    ones = np.ones_like(plain[1][0][..., :1]) * np.ones(d)   # P 2^exponent: at most its sum over the tokens
    top = ref.attend(Q.double().cpu().numpy(), *plain[0], ones, plain[1][1], np.array(table), lens, [M] * B, causal)[0]
    lost = n * 448 * 2.0 ** -40 * top if few else 0
    err = np.abs(O - o)
    assert (err <= w[..., None] * A + 2.0 ** -8 * np.abs(o) + 2.0 ** -134 + lost).all(), (np.argwhere(np.isnan(O))[:3], err.max(), np.abs(o).max())
    err = np.abs(LSE - lse)
    assert (err <= es + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse)).all(), err.max()


def pool(rng, d, ek=-8, ev=-8):
    pages, _ = random_pool(rng, 9, 2, 64, d)
    pages.k_exp.fill_(ek)
    pages.v_exp.fill_(ev)
    return pages, [[8, 2, 3, 0, 7, 5, 1, 4, 6]]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("M", FEW)
@pytest.mark.parametrize("n", [300, 570])       # pages of one CTA a segment, and of more
@pytest.mark.parametrize("ev", [-130, -119, -112, 100, 118])
def test_small_and_large_values_few_rows(d, M, n, ev):
    rng = np.random.default_rng(M + n)
    pages, table = pool(rng, d, ev=ev)
    table = [table[0][: -(-n // 64)]]
    Q = bf16(rng, 1, 2, M, d)
    check(Q, run(Q, pages, table, [n]), plain_of(pages), table, [n])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("M", MANY)
@pytest.mark.parametrize("ev", [-124, -119, -110, 100, 110])   # (sums of values near 2^128 overflow, as the forward's do)
def test_small_and_large_values_many_rows(d, M, ev):
    rng = np.random.default_rng(M)
    pages, table = pool(rng, d, ev=ev)
    Q = bf16(rng, 1, 2, M, d)
    check(Q, run(Q, pages, table, [570]), plain_of(pages), table, [570], few=False)


@pytest.mark.parametrize("M", FEW + MANY)
@pytest.mark.parametrize("ev", [143, 200, 250])
def test_channels_of_zeros_beside_values_past_fp32(M, ev):
    """Values of 2^ev have no bf16; a channel whose codes are all zero is zero all the same."""
    rng = np.random.default_rng(M)
    pages, table = pool(rng, 64, ev=ev)
    pages.v_codes[..., 10:20] = 0
    Q = bf16(rng, 1, 2, M, 64)
    O, LSE = run(Q, pages, table, [570])
    assert (O[..., 10:20] == 0).all() and torch.isfinite(LSE).all()
    if M in FEW:
        o = ref.attend(Q.double().cpu().numpy(), *plain_of(pages)[0], *plain_of(pages)[1], np.array(table), [570], [M], True)[0]
        far = np.abs(o) > 2.0 ** 128
        got = O.double().cpu().numpy()
        assert far.sum() > M * 64 and np.array_equal(got[far], np.copysign(np.inf, o[far]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("M", FEW + MANY)
def test_large_appended_value_that_a_row_does_not_see(d, M):
    """A finite bf16 value appended as 256 * 2^120 = 2^128: rows before it are as if it were zero, rows that see
    it have a finite result."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(d + M)
    L, block = 512 + M, 64
    pages, _ = random_pool(rng, 12, 2, block, d)
    table = [list(range(12))]
    u = L - M + M // 2   # seen by query tokens M // 2 and later
    pages.v_exp[u // block] = 120
    pages.v_codes[u // block] = 0
    Q = bf16(rng, 1, 2, M, d)
    clean = run(Q, pages, table, [L])
    if u % block == 0:   # (append finds the page empty)
        pages.v_exp[u // block] = -160
    V = torch.zeros(1, 2, 1, d, dtype=torch.bfloat16, device="cuda")
    V[..., 3], V[..., 40] = 3.3e38, -3.35e38
    K = bf16(rng, 1, 2, 1, d)
    keep = [t.clone() for t in pages[:2]]
    fv.check_status(fv.fvattn_cache_append(K, V, pages, i32(table), i32([u])), "append")
    for a, b in zip(pages[:2], keep):
        a.copy_(b)
    assert (pages.v_exp[u // block] == 120).all() and (pages.v_codes[u // block, :, u % block, 3] == CODE_256).all()
    got = run(Q, pages, table, [L])
    assert torch.equal(got[0][:, :, : M // 2], clean[0][:, :, : M // 2]) and torch.equal(got[1], clean[1])
    plain = plain_of(pages)
    if M in MANY:
        plain[1][0][np.abs(plain[1][0]) * 2.0 ** plain[1][1][..., None, None].astype(float) >= 2.0 ** 128] *= 255 / 256
    check(Q, got, plain, table, [L], few=M in FEW)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("M", FEW + MANY)
def test_keys_of_2_128_and_small_queries(d, M):
    """Keys at the upper end, queries so small that the scores are ordinary numbers."""
    rng = np.random.default_rng(d + M)
    pages, table = pool(rng, d, ek=120)
    pages.k_codes.bitwise_and_(0x87)            # up to 2^-6 of the scale, but for
    pages.k_codes[:, :, ::7, 5] = CODE_256      # these
    Q = bf16(rng, 1, 2, M, d) * 2.0 ** -118
    plain = plain_of(pages)
    if M in MANY:
        plain[0][0][plain[0][0] == 256] = 255
    check(Q, run(Q, pages, table, [570]), plain, table, [570], few=M in FEW)


@pytest.mark.parametrize("M", FEW + MANY)
def test_large_queries_and_keys_in_different_channels(M):
    """Products that are zero, whose scales multiply to more than fp32 holds."""
    rng = np.random.default_rng(M)
    pages, table = pool(rng, 64, ek=110)
    pages.k_codes[..., :32] = 0
    Q = bf16(rng, 1, 2, M, 64) * 2.0 ** 110
    Q[..., 32:] = 0
    check(Q, run(Q, pages, table, [570]), plain_of(pages), table, [570], few=M in FEW)
    # one channel in common, with small keys: scores of ordinary size
    pages, table = pool(rng, 64, ek=-113)
    pages.k_codes[..., :31] = 0
    Q = bf16(rng, 1, 2, M, 64) * 2.0 ** 110
    Q[..., 32:] = 0
    pages.k_codes[..., 32:] = 0
    check(Q, run(Q, pages, table, [570]), plain_of(pages), table, [570], few=M in FEW)
