"""The paged 8-bit cache on the GPU: append and attention against the 64-bit formulas.

Bounds (u = half a step: fp32 2^-24, fp16 2^-11, bf16 2^-8, e4m3 2^-4 relative, 2^-10 of the
scale below 2^-6):
  append   |code 2^e - x| <= max(2^-4 |x|, 2^-10 2^e) + 6e-7 (|x_a| + |x_b|) (the rotation's fp32
           error, see test_rope_gpu.py); an exponent may differ by one only where the largest
           magnitude is within that error of a power of two times 448.
  attend   score error e_s = (d + 16) 2^-24 sum |q||k| / sqrt(d) (fp32 sums, scale, argument of
           the exponential); a weight's relative error w = 2^-11 (fp16, up to 32 rows; here
           2^-8 above) or 2^-8 (bf16) + 2 e_s + 2^-20 (exponentials and their rescaling) + n 2^-24 (fp32 sums over n
           tokens); |dO| <= w sum P|v| + 2^-8 |O|; |dLSE| <= e_s + 2^-20 + n 2^-24 + 2^-22 |LSE|."""
import numpy as np
import pytest
import torch

from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

ANGLE = 6e-7


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def i32(x):
    return dev(np.asarray(x, dtype=np.int32), torch.int32)


def random_pool(rng, pages, H, block, d, spread=3):
    """A pool as KvPages and as numpy (code values, exponents) pairs; exponents differ by `spread`."""
    import top_routed_block_b200 as fv
    out, plain = [], []
    for _ in range(2):
        x = np.clip(rng.standard_normal((pages, H, block, d)) * 90, -448, 448)
        codes = torch.from_numpy(ref.round_e4m3(x)).float().to(torch.float8_e4m3fn).view(torch.uint8)
        exps = rng.integers(-8, -8 + spread, (pages, H)).astype(np.int32)
        out += [codes.cuda(), dev(exps, torch.int32)]
        plain.append([ref.VALUES[codes.numpy()], exps.copy()])
    return fv.KvPages(*out), plain


def random_table(rng, pages, B, per_seq):
    return rng.permutation(pages)[: B * per_seq].reshape(B, per_seq).astype(np.int32)


def bf16(rng, *shape, layout="bhnd"):
    B, H, n, d = shape
    if layout == "bhnd":
        return dev(rng.standard_normal(shape), torch.bfloat16)
    return dev(rng.standard_normal((B, n, H, d)), torch.bfloat16).transpose(1, 2)


# ------------------------------------------------------------------ append


def check_pool(pages, plain, exact_v=True, size_k=None):
    """Codes and exponents of the pool against the plain form's (code units, unrounded new values)."""
    for i, (codes, exps) in enumerate(((pages.k_codes, pages.k_exp), (pages.v_codes, pages.v_exp))):
        want, e = plain[i]
        got_e = exps.cpu().numpy()
        got = ref.VALUES[codes.cpu().numpy()]
        assert np.array_equal(got_e, e), np.argwhere(got_e != e)[:4]
        if i == 1 and exact_v:
            r = ref.round_e4m3(want)
            assert np.array_equal(np.isnan(got), np.isnan(r))
            assert np.array_equal(got[~np.isnan(r)], r[~np.isnan(r)])
        else:
            clip = np.clip(want, -448, 448)
            tol = np.maximum(2.0 ** -4 * np.abs(clip), 2.0 ** -10) + (0 if size_k is None else size_k)
            bad = ~(np.abs(got - clip) <= tol) & ~(np.isnan(got) & np.isnan(want))
            assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("d,block", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,H,T,starts,new,rope", [
    (1, 1, 1, [0], None, None),
    (3, 2, 1, [5, 127, 128], None, "interleaved"),
    (2, 3, 200, [61, 300], [200, 7], "half"),
    (4, 2, 65, [0, 64, 63, 190], [0, 65, 1, 64], "interleaved"),
    (1, 2, 513, [1], None, None),
])
def test_append(d, block, B, H, T, starts, new, rope):
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(d + block + T)
    per_seq = -(-(max(starts) + T) // block)
    n_pages = B * per_seq + 2
    pages, plain = random_pool(rng, n_pages, H, block, d)
    before = [t.clone() for t in pages]
    table = random_table(rng, n_pages, B, per_seq)
    K, V = bf16(rng, B, H, T, d, layout="bnhd"), bf16(rng, B, H, T, d)
    K.mul_(dev(2.0 ** rng.integers(-6, 7, (B, 1, T, 1)), torch.bfloat16))   # some pages' scales grow, some do not
    pos = rng.integers(0, 5000, (B, T, 2)).astype(np.int32) if rope else None
    axes = fv.rope_axes((d // 2, d // 4), pairing=rope) if rope else None
    st = fv.fvattn_cache_append(K, V, pages, i32(table), i32(starts), new_lens=None if new is None else i32(new),
                                positions=None if pos is None else i32(pos), rope=axes)
    fv.check_status(st, "append")
    new = [T] * B if new is None else new
    k, size = K.double().cpu().numpy(), None
    if rope:
        size = np.stack([ref.partner_size(k[b], len(axes.inv_freq), rope) for b in range(B)])
        k = np.stack([ref.turn(k[b], pos[b], axes.inv_freq, axes.pair_axis, rope) for b in range(B)])
    ref.append(plain, table, starts, new, k, V.double().cpu().numpy())
    err = None
    if rope:  # the rotation's error, in code units where the new keys went
        err = [np.zeros_like(plain[0][0]), plain[0][1].copy()]
        for b in range(B):
            for t in range(new[b]):
                pg, slot = divmod(starts[b] + t, block)
                page = table[b, pg]
                err[0][page, :, slot] = ANGLE * size[b, :, t] * 2.0 ** -plain[0][1][page].astype(float)[:, None]
        err = err[0]
    check_pool(pages, plain, size_k=err)
    # what no new token and no grown scale reaches is left as it was
    for b in range(B):
        for t in range(starts[b] + new[b], per_seq * block):
            pg, slot = divmod(t, block)
            for i in (0, 2):
                assert torch.equal(pages[i][table[b, pg], :, slot], before[i][table[b, pg], :, slot])
    unused = sorted(set(range(n_pages)) - set(table.flatten().tolist()))
    for a, b_ in zip(pages, before):
        assert torch.equal(a[unused], b_[unused])
    # the same tokens at the same place again: the same pool
    snap = [t.clone() for t in pages]
    fv.fvattn_cache_append(K, V, pages, i32(table), i32(starts), new_lens=i32(new),
                           positions=None if pos is None else i32(pos), rope=axes)
    assert all(torch.equal(a, b_) for a, b_ in zip(pages, snap))


def test_append_to_empty_pages_is_the_quantizer(oracle_mod):
    """Without positions and from an empty page on: byte for byte what the quantizer gives."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(3)
    B, H, N, d, block = 1, 3, 384, 128, 128
    pages, _ = random_pool(rng, 3, H, block, d)
    K, V = bf16(rng, B, H, N, d), bf16(rng, B, H, N, d)
    V[0, 1, 128:256] *= 1e-20
    st = fv.fvattn_cache_append(K, V, pages, i32([[0, 1, 2]]), i32([0]))
    fv.check_status(st)
    for x, codes, exps in ((K, pages.k_codes, pages.k_exp), (V, pages.v_codes, pages.v_exp)):
        c, e = fv.fvattn_quant_e4m3(x, block)
        assert torch.equal(codes.transpose(0, 1).reshape(1, H, N, d), c)
        assert torch.equal(exps.t().reshape(1, H, 3), e)


def test_append_zeros_infinities_and_nan():
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(5)
    pages, plain = random_pool(rng, 2, 1, 64, 64)
    table = np.array([[1, 0]], dtype=np.int32)
    steps = [torch.zeros(1, 1, 3, 64), torch.randn(1, 1, 2, 64) * 1e-3, torch.zeros(1, 1, 1, 64),
             torch.full((1, 1, 1, 64), float("nan")), torch.randn(1, 1, 4, 64) * 1e5,
             torch.full((1, 1, 1, 64), float("inf")), torch.randn(1, 1, 70, 64) * 1e-30]
    at = 0
    for x in steps:
        x = x.to(torch.bfloat16).cuda()
        st = fv.fvattn_cache_append(x, x, pages, i32(table), i32([at]))
        fv.check_status(st)
        xn = x.double().cpu().numpy()
        ref.append(plain, table, [at], [x.shape[2]], xn, xn)
        for p in plain:
            p[0] = ref.round_e4m3(p[0])
        at += x.shape[2]
        check_pool(pages, plain)
    assert int(pages.k_exp[1, 0]) == plain[0][1][1, 0]


def test_append_bad_pages_and_starts():
    """Entries outside the pool, starts and counts outside their ranges: reported, left out, and the
    other sequences appended."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(7)
    H, block, d, T = 2, 64, 64, 10
    for starts, new, table, good in [
        ([0, 3, 0], None, [[0, 1], [-1, 2], [3, 4]], [0, 2]),
        ([0, 3, 0], None, [[0, 1], [6, 2], [3, 4]], [0, 2]),
        ([-1, 3, 0], None, [[0, 1], [5, 2], [3, 4]], [1, 2]),
        ([2 ** 31 - 1, 3, 0], None, [[0, 1], [5, 2], [3, 4]], [1, 2]),
        ([0, 3, 0], [10, 11, -4], [[0, 1], [5, 2], [3, 4]], [0]),
    ]:
        pages, plain = random_pool(rng, 6, H, block, d)
        before = [t.clone() for t in pages]
        K, V = bf16(rng, 3, H, T, d), bf16(rng, 3, H, T, d)
        st = fv.fvattn_cache_append(K, V, pages, i32(table), i32(starts), new_lens=None if new is None else i32(new))
        with pytest.raises(fv.FvattnError) as e:
            fv.check_status(st)
        assert e.value.status == fv.FVATTN_ERR_BAD_PAGE
        for b in good:
            ref.append(plain, np.array(table[b: b + 1]), starts[b: b + 1], [T], K[b: b + 1].double().cpu().numpy(),
                       V[b: b + 1].double().cpu().numpy())
        if new is None:
            check_pool(pages, plain)
        # past the table's end: only what fits
    pages, plain = random_pool(rng, 2, H, block, d)
    K, V = bf16(rng, 1, H, T, d), bf16(rng, 1, H, T, d)
    st = fv.fvattn_cache_append(K, V, pages, i32([[1]]), i32([60]))
    with pytest.raises(fv.FvattnError):
        fv.check_status(st)
    ref.append(plain, np.array([[1]]), [60], [4], K.double().cpu().numpy(), V.double().cpu().numpy())
    check_pool(pages, plain)


# ------------------------------------------------------------------ attention


def check_attend(O, LSE, want, new, n_tokens, rows, d):
    o, lse, A, S = want
    o, lse = o.copy(), lse.copy()
    es = (d + 16) * 2.0 ** -24 * S
    w = (2.0 ** -11 if rows <= 32 else 2.0 ** -8) + 2 * es + 2.0 ** -20 + n_tokens * 2.0 ** -24
    got, got_l = O.double().cpu().numpy(), LSE.double().cpu().numpy()
    for b, n in enumerate(new):
        assert np.isfinite(got[b, :, :n]).all()
        err = np.abs(got[b, :, :n] - o[b, :, :n])
        tol = w[b, :, :n, None] * A[b, :, :n] + 2.0 ** -8 * np.abs(o[b, :, :n])
        assert (err <= tol).all(), (b, np.argwhere(err > tol)[:3], err.max())
        empty = np.isneginf(lse[b, :, :n])
        assert np.array_equal(np.isneginf(got_l[b, :, :n]), empty) and not np.isnan(got_l[b, :, :n]).any()
        assert (got[b, :, :n][empty] == 0).all()
        fin = ~empty
        err = np.abs(got_l[b, :, :n][fin] - lse[b, :, :n][fin])
        assert (err <= es[b, :, :n][fin] + 2.0 ** -20 + n_tokens * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse[b, :, :n][fin])).all()


def attend_case(rng, B, H, G, M, d, block, lens, new, causal, spread=3, spoil=True, q_scale=1.0, k_exp=None):
    import top_routed_block_b200 as fv
    per_seq = max(1, -(-max(lens) // block))
    n_pages = B * per_seq + 1
    pages, plain = random_pool(rng, n_pages, H, block, d, spread)
    table = random_table(rng, n_pages, B, per_seq)
    if k_exp is not None:  # one scale for all keys
        pages.k_exp.fill_(k_exp)
        plain[0][1][:] = k_exp
    if spoil:  # behind a sequence's end: NaN codes; and table entries that no token uses name no page
        for b in range(B):
            for t in range(lens[b], per_seq * block):
                pg, slot = divmod(t, block)
                pages.k_codes[table[b, pg], :, slot] = 0x7F
                pages.v_codes[table[b, pg], :, slot] = 0xFF
            table[b, -(-lens[b] // block):] = -7 if b % 2 else 1 << 30
    Q = (bf16(rng, B, H * G, M, d, layout="bnhd") * q_scale)
    O = torch.full((B, M, H * G, d), 3.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    LSE = torch.full((B, H * G, M), 5.0, device="cuda")
    args = (Q, pages, i32(table), i32(lens))
    _, _, st = fv.fvattn_cache_attend(*args, new_lens=None if new is None else i32(new), causal=causal, O=O, LSE=LSE)
    fv.check_status(st, "attend")
    nw = [M] * B if new is None else new
    want = ref.attend(Q.double().cpu().numpy(), plain[0][0], plain[0][1], plain[1][0], plain[1][1], table, lens, nw, causal)
    check_attend(O, LSE, want, nw, max(lens), G * M, d)
    for b, n in enumerate(nw):  # rows behind a sequence's new tokens
        assert (O[b, :, n:] == 3).all() and (LSE[b, :, n:] == 5).all()
    return args, O, LSE


@pytest.mark.parametrize("d,block", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,H,G,M,lens,new,causal", [
    (1, 1, 1, 1, [1], None, True),
    (1, 2, 1, 1, [0], None, False),
    (3, 2, 1, 1, [129, 1, 640], None, True),
    (2, 1, 4, 2, [100, 31], None, True),
    (2, 2, 3, 5, [33, 700], [5, 2], True),          # 15 rows, two row groups
    (3, 1, 2, 7, [3, 0, 515], [7, 0, 6], True),     # more new tokens than cached ones: rows that see nothing
    (2, 1, 8, 4, [257, 64], None, False),           # 32 rows
    (2, 2, 1, 33, [300, 40], None, True),           # tiles of 128 rows from here on
    (2, 1, 5, 29, [129, 513], [29, 3], True),       # a tile over several heads' rows
    (3, 1, 1, 130, [128, 0, 255], [130, 0, 128], True),
    (1, 2, 1, 257, [1000], None, False),
    (2, 3, 2, 33, [600, 2049], None, True),         # 66 rows: one tile, cut over its keys
    (2, 2, 1, 64, [1500, 700], [64, 9], True),      # 64 rows: eight row groups
    (1, 1, 1, 70, [512], None, True),               # a short cache: a CTA takes all of it
    (1, 150, 1, 129, [700], None, True),            # more items than SMs: whole ones, then the rest
])
def test_attend(d, block, B, H, G, M, lens, new, causal):
    attend_case(np.random.default_rng(M * 7 + d + block), B, H, G, M, d, block, lens, new, causal)


@pytest.mark.parametrize("G,M,n", [(1, 1, 40000), (2, 3, 9001), (1, 1, 128 * 300)])
def test_attend_long_split(G, M, n):
    """Enough tokens for many chunks each of many warps."""
    attend_case(np.random.default_rng(n), 1, 1, G, M, 128, 128, [n], None, True, spoil=n < 10000)


@pytest.mark.parametrize("M", [1, 40, 130])
def test_attend_scales_far_apart(M):
    """Pages whose scales differ by 2^40, and scores in the hundreds: weights of a page with small values
    must not be lost beside those of a page with large ones that the softmax has all but removed."""
    rng = np.random.default_rng(31)
    attend_case(rng, 2, 2, 1, M, 64, 64, [500, 300], None, False, spread=40, q_scale=0.05)
    attend_case(rng, 2, 2, 1, M, 128, 128, [500, 300], None, True, q_scale=12.0)
    for q_scale in (0.3, 2.0):
        attend_case(rng, 2, 2, 1, M, 64, 64, [500, 300], None, False, spread=40, q_scale=q_scale, k_exp=-7)


@pytest.mark.parametrize("M", [5, 70, 150])
def test_attend_nan_that_a_row_does_not_see(M):
    """Causal rows around a cached token with a NaN value (one channel) and a NaN key: rows before it are
    as if it were not there, rows that see the value have NaN in that channel only."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(37)
    d, block, L = 64, 64, 200
    pages, plain = random_pool(rng, 4, 1, block, d)
    table = np.arange(4, dtype=np.int32)[None]
    Q = bf16(rng, 1, 1, M, d)
    u = L - M + 2   # seen by query tokens 2 and later
    clean = fv.fvattn_cache_attend(Q, pages, i32(table), i32([L]), causal=True)[:2]
    pages.v_codes[u // block, 0, u % block, 9] = 0x7F
    O, LSE, st = fv.fvattn_cache_attend(Q, pages, i32(table), i32([L]), causal=True)
    fv.check_status(st)
    assert torch.equal(O[:, :, :2], clean[0][:, :, :2]) and torch.equal(LSE, clean[1])
    bad = torch.isnan(O[0, 0])
    assert bad[2:, 9].all() and bad.sum() == M - 2
    keep = [c for c in range(d) if c != 9]
    assert torch.equal(O[..., keep], clean[0][..., keep])
    # a NaN key: the rows that see it are NaN throughout, LSE too
    pages.k_codes[u // block, 0, u % block, 3] = 0xFF
    O, LSE, st = fv.fvattn_cache_attend(Q, pages, i32(table), i32([L]), causal=True)
    assert torch.equal(O[:, :, :2], clean[0][:, :, :2]) and torch.equal(LSE[..., :2], clean[1][..., :2])
    assert torch.isnan(O[:, :, 2:]).all() and torch.isnan(LSE[..., 2:]).all()


@pytest.mark.parametrize("M", [2, 50, 200])
def test_attend_bad_pages(M):
    """Table entries and lengths out of range are reported, and read nothing outside the pool."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(41)
    pages, _ = random_pool(rng, 4, 2, 64, 64)
    Q = bf16(rng, 2, 2, M, 64)
    for table, lens, new in [([[0, -1], [2, 3]], [100, 128], None), ([[0, 4], [2, 3]], [100, 128], None),
                             ([[0, 1], [2, 3]], [129, 128], None), ([[0, 1], [2, 3]], [100, -3], None),
                             ([[0, 1], [2, 3]], [100, 128], [M + 1, 1]), ([[0, 1], [2, 3]], [100, 128], [-1, M])]:
        _, _, st = fv.fvattn_cache_attend(Q, pages, i32(table), i32(lens), new_lens=None if new is None else i32(new))
        with pytest.raises(fv.FvattnError) as e:
            fv.check_status(st)
        assert e.value.status == fv.FVATTN_ERR_BAD_PAGE
    _, _, st = fv.fvattn_cache_attend(Q, pages, i32([[0, 1], [2, 3]]), i32([100, 128]))
    fv.check_status(st)


@pytest.mark.parametrize("M", [1, 9, 70])
@pytest.mark.parametrize("B", [3, 70])   # the work of few rows in chunks, in stretches
def test_attend_bad_pages_of_long_tables(B, M):
    """A bad entry anywhere among a sequence's cached tokens is reported, one behind them or of a sequence
    without queries is not; the next good call says so."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(42)
    pages, _ = random_pool(rng, 12, 2, 64, 64)
    Q = bf16(rng, B, 2, M, 64)
    good = rng.integers(0, 12, (B, 11)).astype(np.int32)
    lens = rng.integers(M, 500, B).astype(np.int32)
    lens[1], lens[2] = 11 * 64 - 5, 300
    new = np.full(B, M, np.int32)
    new[2] = 0
    status = torch.empty(1, dtype=torch.int32, device="cuda")
    for (b, pg), bad in [((1, 0), True), ((1, 6), True), ((1, 10), True), ((2, 1), False), ((0, 10), False), ((0, 0), True)]:
        table = good.copy()
        table[b, pg] = 12 if pg else -1
        fv.fvattn_cache_attend(Q, pages, i32(table), i32(lens), new_lens=i32(new), dev_status=status)
        assert int(status) == (fv.FVATTN_ERR_BAD_PAGE if bad else 0), (b, pg)
    fv.fvattn_cache_attend(Q, pages, i32(good), i32(lens), new_lens=i32(new), dev_status=status)
    assert int(status) == 0


@pytest.mark.parametrize("M", [1, 3, 65])
def test_attend_repeats_streams_graphs(M):
    """The same bits again, on another stream, two calls at once, and captured and replayed with other
    lengths and inputs."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(43)
    args, O, LSE = attend_case(rng, 2, 3, 2, M, 128, 64, [2000, 700], None, True, spoil=False)
    Q, pages, table, lens = args
    again = fv.fvattn_cache_attend(*args, causal=True)
    assert torch.equal(again[0], O) and torch.equal(again[1], LSE)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [fv.fvattn_cache_attend(*args, causal=True, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], O) and torch.equal(g[1], LSE) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fv.fvattn_cache_attend(*args, causal=True)
    lens.copy_(i32([701, 1999]))
    Q.copy_(torch.randn_like(Q))
    for _ in range(2):
        graph.replay()
    want = fv.fvattn_cache_attend(*args, causal=True)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_attend_shared_pages():
    """A page in two sequences' tables (a common prefix) is read by both."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(47)
    pages, plain = random_pool(rng, 5, 2, 64, 64)
    table, lens = np.array([[3, 1], [3, 4]], dtype=np.int32), [100, 90]
    Q = bf16(rng, 2, 2, 1, 64)
    O, LSE, st = fv.fvattn_cache_attend(Q, pages, i32(table), i32(lens))
    fv.check_status(st)
    want = ref.attend(Q.double().cpu().numpy(), *plain[0], *plain[1], table, lens, [1, 1], False)
    check_attend(O, LSE, want, [1, 1], 100, 1, 64)


@pytest.mark.parametrize("d,block", [(64, 64), (128, 128)])
def test_generation_run(d, block):
    """A cache filled and read as a program does: a prompt, a ragged chunk, then single tokens, with
    grid positions; each step's attention against the formulas over what the cache then holds, and
    the cached values against the turned inputs."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(53 + d)
    B, H, G = 2, 2, 2
    rope = fv.rope_axes((d // 2, d // 4, d // 4))
    grid = fv.grid_positions(12, 5, 6)
    cache = fv.FvattnCache(B, H, d, block, 360)
    said = [np.zeros((H, 0, d)) for _ in range(B)]
    for T, new in ((150, None), (40, [40, 3]), (1, None), (1, None), (1, [0, 1])):
        lens = cache.lens.tolist()
        K, V = bf16(rng, B, H, T, d, layout="bnhd"), bf16(rng, B, H, T, d)
        Q = bf16(rng, B, H * G, T, d, layout="bnhd")
        pos = torch.stack([grid[n: n + T] for n in lens]).contiguous()
        Qr, _ = fv.fvattn_rope(Q, None, pos, rope)
        nl = None if new is None else i32(new)
        cache.append(K, V, new_lens=nl, positions=pos, rope=rope)
        O = torch.zeros(B, H * G, T, d, dtype=torch.bfloat16, device="cuda")
        LSE = torch.zeros(B, H * G, T, device="cuda")
        cache.attend(Qr, new_lens=nl, O=O, LSE=LSE)
        cache.check()
        nw = [T] * B if new is None else new
        assert cache.lens.tolist() == [a + n for a, n in zip(lens, nw)]
        kv = [ref.VALUES[c.cpu().numpy()] for c in (cache.pages.k_codes, cache.pages.v_codes)]
        ke, ve = cache.pages.k_exp.cpu().numpy(), cache.pages.v_exp.cpu().numpy()
        want = ref.attend(Qr.double().cpu().numpy(), kv[0], ke, kv[1], ve, cache.page_table.cpu().numpy(),
                          cache.lens.tolist(), nw, True)
        check_attend(O, LSE, want, nw, max(cache.lens.tolist()), G * T, d)
        for b in range(B):
            k = ref.turn(K[b].double().cpu().numpy(), pos[b].cpu().numpy(), rope.inv_freq, rope.pair_axis, "interleaved")
            said[b] = np.concatenate([said[b], k[:, : nw[b]]], 1)
    for b in range(B):
        n = said[b].shape[1]
        ids = cache.page_table[b].cpu().numpy()
        got = (kv[0][ids] * 2.0 ** ke[ids].astype(float)[..., None, None]).transpose(1, 0, 2, 3).reshape(H, -1, d)[:, :n]
        step = np.repeat(2.0 ** (ke[ids].astype(float) - 10).T, block, 1)[:, :n, None]
        # one rounding when it came, and one more for each growth of a page's scale that made it subnormal
        assert (np.abs(got - said[b]) <= 2.0 ** -4 * np.abs(said[b]) + 2 * step + 1e-5).all()


def test_attend_wide_batch():
    """More sequences than the planning searches chunks for, most of them short or empty."""
    rng = np.random.default_rng(61)
    lens = [int(x) for x in rng.integers(0, 90, 70)]
    lens[3], lens[40] = 1300, 640
    attend_case(rng, 70, 1, 1, 1, 64, 64, lens, None, True)
    # short caches, a CTA each: more of them than there are SMs
    lens = [int(x) for x in rng.integers(0, 257, 80)]
    attend_case(rng, 80, 2, 2, 1, 64, 64, lens, None, True)
    attend_case(rng, 5, 2, 5, 24, 64, 64, [256, 24, 1, 130, 70], [24, 24, 1, 3, 0], True)


def test_append_many_items():
    """More pages and heads than resident CTAs: stretches that end inside a page's heads."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(67)
    B, H, T, d, block = 2, 23, 1300, 128, 128
    pages, plain = random_pool(rng, 24, H, block, d)
    table, starts = random_table(rng, 24, B, 12), [70, 129]
    K, V = bf16(rng, B, H, T, d, layout="bnhd"), bf16(rng, B, H, T, d, layout="bnhd")
    st = fv.fvattn_cache_append(K, V, pages, i32(table), i32(starts))
    fv.check_status(st)
    ref.append(plain, table, starts, [T] * B, K.double().cpu().numpy(), V.double().cpu().numpy())
    check_pool(pages, plain)


def test_append_on_streams_and_in_a_graph():
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(71)
    for T in (1, 40):
        rope, pos = fv.rope_axes((64,)), i32(np.arange(T)[:, None] + 5)
        table, start = i32([[0, 1], [3, 2]]), i32([5, 70])
        made = [random_pool(rng, 4, 2, 64, 64)[0] for _ in range(3)]
        for m in made[1:]:
            for a, b in zip(m, made[0]):
                a.copy_(b)
        K, V = bf16(rng, 2, 2, T, 64), bf16(rng, 2, 2, T, 64)
        args = dict(positions=pos, rope=rope)
        fv.check_status(fv.fvattn_cache_append(K, V, made[0], table, start, **args))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        st = fv.fvattn_cache_append(K, V, made[1], table, start, stream=s, **args)
        s.synchronize()
        fv.check_status(st)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            st = fv.fvattn_cache_append(K, V, made[2], table, start, **args)
        graph.replay()
        fv.check_status(st)
        for a, b, c in zip(*made):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_attend_refuses_on_the_gpu():
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(59)
    pages, _ = random_pool(rng, 2, 2, 64, 64)
    Q, table, lens = bf16(rng, 1, 2, 1, 64), i32([[0, 1]]), i32([70])
    for bad in (dict(Q=Q[:, :1]), dict(Q=Q.float()), dict(lens=lens.long()), dict(table=table[0]), dict(lens=i32([1, 2])),
                dict(pages=pages._replace(k_exp=pages.k_exp[:, :1])), dict(pages=pages._replace(v_codes=pages.v_codes[:1]))):
        a = dict(Q=Q, pages=pages, table=table, lens=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            fv.fvattn_cache_attend(a["Q"], a["pages"], a["table"], a["lens"])
    with pytest.raises(fv.FvattnError) as e:
        fv.fvattn_cache_attend(Q, pages, table, lens, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == fv.FVATTN_ERR_CAPACITY
    with pytest.raises(ValueError):
        fv.fvattn_cache_append(Q, Q, pages, table, lens, positions=i32([[0]]))


@pytest.mark.parametrize("M", [1, 90])
def test_offsets_past_32_bits(M):
    """Pages behind the pool's first 2^32 bytes, and a table so wide that the expanded pages pass 2^31 elements."""
    import top_routed_block_b200 as fv
    rng = np.random.default_rng(71)
    H, d, block, n_pages = 8, 128, 128, (1 << 32) // (8 * 128 * 128) + 9
    small, _ = random_pool(rng, 4, H, block, d)
    big = fv.KvPages(torch.empty((n_pages, H, block, d), dtype=torch.uint8, device="cuda"),
                     torch.zeros((n_pages, H), dtype=torch.int32, device="cuda"),
                     torch.empty((n_pages, H, block, d), dtype=torch.uint8, device="cuda"),
                     torch.zeros((n_pages, H), dtype=torch.int32, device="cuda"))
    wide = 16400 if M > 64 else 5     # 8 heads * 16400 pages * 128 tokens * 128 channels: past 2^31
    table = np.full((1, wide), n_pages - 1, np.int32)
    table[0, :4] = n_pages - 1 - np.arange(4)
    for s, b in zip(small, big):
        b[n_pages - 4:] = s.flip(0)
    start = i32([300])
    K, V = bf16(rng, 1, H, M, d), bf16(rng, 1, H, M, d)
    for pages, t in ((small, i32([[0, 1, 2, 3]])), (big, i32(table))):
        fv.check_status(fv.fvattn_cache_append(K, V, pages, t, start), "append")
    for s, b in zip(small, big):
        assert torch.equal(b[n_pages - 4:].flip(0), s)
    Q = bf16(rng, 1, H, M, d)
    lens = start + M
    (kv, ke), (vv, ve) = ((ref.VALUES[c.cpu().numpy()], e.cpu().numpy()) for c, e in (small[:2], small[2:]))
    want = ref.attend(Q.double().cpu().numpy(), kv, ke, vv, ve, np.arange(4)[None], [300 + M], [M], True)
    for pages, t in ((small, i32([[0, 1, 2, 3]])), (big, i32(table))):
        O, LSE, st = fv.fvattn_cache_attend(Q, pages, t, lens, causal=True)
        fv.check_status(st, "attend")
        check_attend(O, LSE, want, [M], 300 + M, M, d)
