"""Attention over the 8-bit cache, both kernels held to the rounding of their own weights: fp16, 2^-11, up to 64 rows of
a key head (128 where the page table holds at most 512 tokens), and bf16, 2^-8, above.  Otherwise the bounds
of test_cache_gpu.py.  And page tables wider than what is cached."""
import numpy as np
import pytest
import torch

from tests import cache_ref as ref
from tests.test_cache_gpu import bf16, check_pool, i32, random_pool, random_table

pytestmark = pytest.mark.gpu


def few_rows(rows, max_pages, block):
    return rows <= (128 if max_pages * block <= 512 else 64)


def check(O, LSE, want, new, n_tokens, few, d):
    o, lse, A, S = want
    es = (d + 16) * 2.0 ** -24 * S
    w = (2.0 ** -11 if few else 2.0 ** -8) + 2 * es + 2.0 ** -20 + n_tokens * 2.0 ** -24
    got, got_l = O.double().cpu().numpy(), LSE.double().cpu().numpy()
    for b, n in enumerate(new):
        err = np.abs(got[b, :, :n] - o[b, :, :n])
        assert (err <= w[b, :, :n, None] * A[b, :, :n] + 2.0 ** -8 * np.abs(o[b, :, :n])).all(), (b, err.max())
        some = ~np.isneginf(lse[b, :, :n])
        assert np.array_equal(~np.isneginf(got_l[b, :, :n]), some) and (got[b, :, :n][~some] == 0).all()
        err = np.abs(got_l[b, :, :n][some] - lse[b, :, :n][some])
        assert (err <= es[b, :, :n][some] + 2.0 ** -20 + n_tokens * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse[b, :, :n][some])).all()


@pytest.mark.parametrize("d,block", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,H,G,M,lens,new,wide", [
    (2, 2, 1, 33, [900, 40], None, 0),
    (2, 1, 3, 16, [700, 600], [16, 5], 0),
    (1, 2, 8, 8, [1300], None, 0),
    (2, 2, 1, 64, [1500, 700], [64, 9], 0),
    (1, 1, 1, 65, [512], None, 0),
    (2, 1, 5, 24, [256, 130], [24, 3], 0),
    (1, 2, 1, 128, [500], None, 0),
    (1, 1, 1, 128, [1, ], [1], 0),
    (3, 2, 1, 1, [509, 0, 77], None, 40),      # a table of 40 pages, mostly unused
    (3, 2, 2, 9, [300, 12, 129], [9, 0, 9], 40),
    (2, 1, 1, 100, [300, 129], [100, 50], 40),
    (2, 2, 1, 130, [300, 129], [130, 1], 300),
])
def test_bounds(d, block, B, H, G, M, lens, new, wide):
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(M * 11 + d + block + wide)
    per_seq = max(-(-n // block) for n in lens)
    pages, plain = random_pool(rng, B * per_seq + 1, H, block, d)
    table = random_table(rng, B * per_seq + 1, B, per_seq)
    Q = bf16(rng, B, H * G, M, d, layout="bnhd")
    nw = [M] * B if new is None else new
    want = ref.attend(Q.double().cpu().numpy(), *plain[0], *plain[1], table, lens, nw, True)
    args = dict(new_lens=None if new is None else i32(new), causal=True)
    tables = [table]
    if wide:   # entries that no token uses name no page
        tables.append(np.concatenate([table, np.where(np.arange(B * wide).reshape(B, wide) % 2, -1, 1 << 30)], 1).astype(np.int32))
    for t in tables:
        for b in range(B):
            t[b, -(-lens[b] // block):] = -3
        O, LSE, st = fv.fvattn_cache_attend(Q, pages, i32(t), i32(lens), **args)
        fv.check_status(st, "attend")
        check(O, LSE, want, nw, max(lens), few_rows(G * M, t.shape[1], block), d)


def test_append_counts_out_of_range_are_held_inside():
    """A count above T appends T tokens, one below zero none."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(7)
    for T, starts in ((10, [0, 3, 0]), (1, [63, 64, 5]), (70, [10, 20, 30])):
        pages, plain = random_pool(rng, 6, 2, 64, 64)
        table = [[0, 1], [5, 2], [3, 4]]
        K, V = bf16(rng, 3, 2, T, 64), bf16(rng, 3, 2, T, 64)
        st = fv.fvattn_cache_append(K, V, pages, i32(table), i32(starts), new_lens=i32([T, T + 1, -4]))
        with pytest.raises(fv.FvattnError) as e:
            fv.check_status(st)
        assert e.value.status == fv.FVATTN_ERR_BAD_PAGE
        ref.append(plain, np.array(table), starts, [T, T, 0], K.double().cpu().numpy(), V.double().cpu().numpy())
        check_pool(pages, plain)
