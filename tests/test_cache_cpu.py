"""Host-side checks of the rotary positions and the 8-bit cache: what the entry points
refuse, the workspace sizes, the index arithmetic of the kernels (compiled for the host) and
the plain forms that the GPU tests compare with."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests import cache_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, ALIGNMENT, CAPACITY = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from top_routed_block_b200 import _build
    _build.build()
    import top_routed_block_b200 as fv
    return fv.load_library()


P = ctypes.c_void_p
FAKE = P(16)  # never dereferenced: argument checks fail first


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def freqs(n):
    return (ctypes.c_double * n)(*([1.0] * n)), (ctypes.c_int32 * n)(*([0] * n))


def rope_args(**kw):
    f, a = freqs(kw.get("n_pairs", 32) if 0 < kw.get("n_pairs", 32) < 1000 else 1)
    args = dict(Q=FAKE, qs=strides(0, 64, 64), Qr=FAKE, qrs=strides(0, 64 * 10, 64), qh=2, K=None, ks=None, Kr=None,
                krs=None, kh=0, B=1, N=10, d=64, pos=FAKE, pos_b=0, freq=f, axis=a, n_pairs=32, n_axes=1, pairing=0,
                inverse=0, stream=None)
    args.update(kw)
    return list(args.values())


@pytest.mark.parametrize("change,rc", [
    (dict(Q=None), INVALID), (dict(Qr=None), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(qh=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(n_pairs=0), INVALID), (dict(n_pairs=33), INVALID), (dict(n_axes=0), INVALID), (dict(n_axes=5), UNSUPPORTED),
    (dict(pairing=2), INVALID), (dict(pairing=1, n_pairs=12), UNSUPPORTED), (dict(inverse=2), INVALID),
    (dict(kh=1), INVALID), (dict(K=FAKE), INVALID), (dict(pos_b=7), INVALID), (dict(Q=P(18)), ALIGNMENT),
    (dict(qs=strides(0, 4, 64)), ALIGNMENT), (dict(qs=strides(0, -64, 64)), INVALID),
    (dict(qrs=strides(0, 0, 64)), INVALID),          # every head written to one place
    (dict(qrs=strides(0, 64, 64)), INVALID),         # rows of two heads overlap
    (dict(B=70000), UNSUPPORTED),
    (dict(Qr=P(4096), K=FAKE, ks=strides(0, 640, 64), Kr=FAKE, krs=strides(0, 64, 64), kh=1, N=1, qh=1, Q=P(8192),
          qs=strides(0, 64, 64)), None),             # (in place with one head and token: nothing to refuse)
    (dict(qrs=strides(0, 640, 64), qs=strides(0, 64, 128)), INVALID),   # in place with other strides
    (dict(Q=P(4096), Qr=P(8192), K=P(8192), ks=strides(0, 64, 64), Kr=P(16), krs=strides(0, 640, 64), kh=2), INVALID),
    (dict(Q=P(4096), Qr=P(8192), K=P(16384), ks=strides(0, 64, 64), Kr=P(8192), krs=strides(0, 640, 64), kh=2), INVALID),
])
def test_rope_refuses(lib, change, rc):
    import torch
    if rc is None and torch.cuda.is_available():
        pytest.skip("would run")
    got = lib.fvattn_rope(*rope_args(**change))
    assert got == rc if rc is not None else got not in (INVALID, ALIGNMENT)


def test_rope_refuses_bad_pairs(lib):
    f, a = freqs(32)
    f[3] = float("nan")
    assert lib.fvattn_rope(*rope_args(freq=f)) == INVALID
    f[3] = 1.0
    for bad in (-1, 1):
        a[5] = bad
        assert lib.fvattn_rope(*rope_args(freq=f, axis=a)) == INVALID


def append_args(**kw):
    f, a = freqs(32)
    args = dict(K=FAKE, ks=strides(0, 64, 64), V=FAKE, vs=strides(0, 64, 64), B=1, heads=2, T=5, d=64, block=64,
                kc=FAKE, ke=FAKE, vc=FAKE, ve=FAKE, num_pages=4, table=FAKE, max_pages=2, start=FAKE, new=None,
                pos=None, pos_b=0, freq=f, axis=a, n_pairs=32, n_axes=1, pairing=0, status=FAKE, stream=None)
    args.update(kw)
    return list(args.values())


@pytest.mark.parametrize("change,rc", [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(kc=None), INVALID), (dict(ve=None), INVALID),
    (dict(table=None), INVALID), (dict(start=None), INVALID), (dict(status=None), INVALID), (dict(T=0), INVALID),
    (dict(B=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(d=32), UNSUPPORTED),
    (dict(block=16), UNSUPPORTED), (dict(kc=P(24)), ALIGNMENT), (dict(ks=strides(0, 4, 64)), ALIGNMENT),
    (dict(max_pages=1 << 24), UNSUPPORTED), (dict(pos=FAKE, n_pairs=33), INVALID), (dict(pos=FAKE, pos_b=3), INVALID),
    (dict(B=1 << 20, heads=1 << 10), UNSUPPORTED),
])
def test_append_refuses(lib, change, rc):
    assert lib.fvattn_cache_append(*append_args(**change)) == rc


def attend_args(**kw):
    args = dict(Q=FAKE, qs=strides(0, 64, 64), B=1, heads=2, group=1, M=1, d=64, block=64, kc=FAKE, ke=FAKE, vc=FAKE,
                ve=FAKE, num_pages=4, table=FAKE, max_pages=2, lens=FAKE, new=None, causal=0, O=FAKE,
                os=strides(0, 64, 64), LSE=FAKE, ws=FAKE, ws_bytes=1 << 40, status=FAKE, stream=None)
    args.update(kw)
    return list(args.values())


@pytest.mark.parametrize("change,rc", [
    (dict(Q=None), INVALID), (dict(O=None), INVALID), (dict(LSE=None), INVALID), (dict(lens=None), INVALID),
    (dict(ws=None), INVALID), (dict(status=None), INVALID), (dict(table=None), INVALID), (dict(M=0), INVALID),
    (dict(group=0), INVALID), (dict(causal=2), INVALID), (dict(d=96), UNSUPPORTED), (dict(block=32), UNSUPPORTED),
    (dict(B=4097), UNSUPPORTED), (dict(max_pages=1 << 25), UNSUPPORTED), (dict(O=P(24)), ALIGNMENT),
    (dict(Q=P(24)), ALIGNMENT), (dict(qs=strides(0, 3, 64)), ALIGNMENT), (dict(os=strides(0, 0, 64)), INVALID),
    (dict(O=FAKE), INVALID),   # where Q lies
    (dict(ws_bytes=64), CAPACITY), (dict(M=100, ws_bytes=64, os=strides(0, 6400, 64)), CAPACITY),
])
def test_attend_refuses(lib, change, rc):
    assert lib.fvattn_cache_attend(*attend_args(**change)) == rc


def test_attend_workspace(lib):
    import top_routed_block_b200 as fv
    ws = fv.fvattn_cache_attend_workspace_bytes
    assert ws(0, 1, 1, 1, 64, 64, 1) == 0 and ws(1, 1, 1, 1, 96, 64, 1) == 0 and ws(4097, 1, 1, 1, 64, 64, 1) == 0
    # more than 64 rows: K and V of every page as bf16
    assert ws(2, 3, 8, 9, 128, 128, 5) >= 2 * 2 * 3 * 5 * 128 * 128 * 2
    # few rows: bounded by the grid, not by the cache's length
    assert 0 < ws(1, 8, 1, 1, 128, 128, 1 << 20) < 64 << 20
    assert 0 < ws(1, 1, 1, 1, 64, 64, 1) < 8 << 20


def test_status_of_bad_pages():
    import top_routed_block_b200 as fv
    assert fv.status_string(fv.FVATTN_ERR_BAD_PAGE) not in ("", "unknown status")


INDEX_CHECK = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "cache_index.h"
using namespace fvattn;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
    // every new token gets one slot of one touched page, and no other slot is named
    for (int block : {64, 128})
        for (long start = 0; start < 400; start += 7)
            for (long T = 1; T < 400; T += 13)
                for (long n : {0L, 1L, T / 2, T}) {
                    const long cap = 6 * block;
                    const long count = append_count(start, n, T, cap);
                    CHECK(count >= 0 && count <= n && (count == 0 || start + count <= cap));
                    std::vector<int> hit(cap, 0);
                    for (long j = 0; j < max_touched_pages(T, block); ++j) {
                        const long pg = start / block + j;
                        const PageSpan s = page_span(start, count, pg, block);
                        if (s.lo >= s.hi) continue;
                        CHECK(s.lo >= 0 && s.hi <= block && pg * block + s.hi <= cap);
                        CHECK(s.token >= 0 && s.token + (s.hi - s.lo) <= count);
                        for (int k = s.lo; k < s.hi; ++k) {
                            CHECK(pg * block + k == start + s.token + (k - s.lo));
                            ++hit[pg * block + k];
                        }
                    }
                    for (long u = 0; u < cap; ++u) CHECK(hit[u] == (u >= start && u < start + count));
                }
    CHECK(append_count(-1, 5, 5, 100) == 0 && append_count(101, 5, 5, 100) == 0 && append_count(98, 5, 5, 100) == 2);
    CHECK(append_count(3, -2, 5, 100) == 0 && append_count(3, 9, 5, 100) == 5 && append_count(2147483647L, 1, 1, 100) == 0);
    CHECK(checked_page(-1, 4) < 0 && checked_page(4, 4) < 0 && checked_page(3, 4) == 3 && checked_page(0, 4) == 0);
    CHECK(checked_page(-2147483647 - 1, 4) < 0 && checked_page(2147483647, 4) < 0);
    CHECK(clamp_len(-5, 10) == 0 && clamp_len(11, 10) == 10 && clamp_len(10, 10) == 10);
    // the plan: the stretches tile the line of units, each unit is found in its own, and a stretch
    // holds at most two segments that are not whole in it
    std::srand(7);
    for (int it = 0; it < 3000; ++it) {
        const int B = 1 + std::rand() % 20;
        const long groups = 1 + std::rand() % 90, ctas = 1 + std::rand() % 443;
        std::vector<long> ends;
        long total = 0;
        for (int b = 0; b < B; ++b) {
            const long len = std::rand() % 4 ? std::rand() % 3000 : 0, u = segment_units(len, 128);
            CHECK(u >= 1 && u * 128 >= len && (u - 1) * 128 < (len > 0 ? len : 1));
            for (long k = 0; k < groups; ++k) ends.push_back(total += u);
        }
        const long n = stretches(total, ctas);
        CHECK(n >= 1 && n <= ctas);
        CHECK(stretch_start(0, total, n) == 0 && stretch_start(n, total, n) == total);
        for (long c = 0; c < n; ++c) {
            const long s0 = stretch_start(c, total, n), s1 = stretch_start(c + 1, total, n);
            CHECK(s0 < s1);
            for (long u = s0; u < s1; ++u) CHECK(stretch_of(u, total, n) == c);
        }
        long from = 0;
        std::vector<int> begun(n, 0), carried(n, 0);
        for (long end : ends) {
            const int c0 = stretch_of(from, total, n), c1 = stretch_of(end - 1, total, n);
            if (c0 != c1) {
                ++begun[c0];
                for (int c = c0 + 1; c <= c1; ++c) ++carried[c];
            }
            from = end;
        }
        for (long c = 0; c < n; ++c) CHECK(begun[c] <= 1 && carried[c] <= 1);
    }
    return 0;
}
"""


def test_index_arithmetic(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "index.cpp"
    src.write_text(INDEX_CHECK)
    exe = tmp_path / "index"
    inc = os.path.join(ROOT, "top_routed_block_b200", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", inc, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def chunk_place(d, row, at):
    """Where the few-rows kernel keeps byte `at` of a row in shared memory."""
    byte = row * d + at
    line = byte >> 7
    mix = (((line >> 1) & 3) << 1) ^ ((line & 1) << 2) if d == 128 else (line & 3) << 1
    return (line << 7) + ((((byte >> 4) & 7) ^ mix) << 4) + (byte & 8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [32, 64])
def test_lanes_read_each_cached_byte_once(d, step):
    """The few-rows kernel: the copies write every place once, the lanes read every byte once in the
    order of the products, and no two lanes of a quarter (half) warp meet in a bank."""
    places = sorted(chunk_place(d, r, c) + i for r in range(step) for c in range(0, d, 8) for i in range(8))
    assert places == list(range(step * d))

    def check(reads, size):
        hit = np.zeros(step * d, int)
        for r in reads:   # one instruction: (row, byte) of each lane
            for lo in range(0, 32, 128 // size):
                banks = [(chunk_place(d, *x) // 4 + w) % 32 for x in r[lo: lo + 128 // size] for w in range(size // 4)]
                assert len(set(banks)) == len(banks)
            for row, at in r:
                assert at % size == 0
                hit[row * d + at: row * d + at + size] += 1
        assert (hit == 1).all()

    lanes = [(lane >> 2, lane & 3) for lane in range(32)]
    # the places as a lane's constant and an immediate
    for lane, (g, q) in enumerate(lanes):
        line = lane >> 3
        c = chunk_place(d, line * 128 // d, (lane & 7) * 16 % d) if d == 128 else chunk_place(
            d, line * 2 + (lane & 7) // 4, (lane & 3) * 16)
        for i in range(step * d // 512):
            byte = i * 512 + lane * 16
            assert (c ^ 64 if d == 128 and i & 1 else c) + i * 512 == chunk_place(d, byte // d, byte % d)
        k, v = chunk_place(d, g, q * 16), chunk_place(d, 2 * q, g * (d // 8))
        for r8 in range(step // 8):
            for half in range(d // 64):
                assert (k ^ 64 if half else k) + r8 * 8 * d == chunk_place(d, g + 8 * r8, half * 64 + q * 16)
            for odd in range(2):
                want = chunk_place(d, 2 * q + odd + 8 * r8, g * (d // 8))
                assert ((v ^ 64) + (128 if d == 128 else 0) if odd else v) + r8 * 8 * d == want
    check([[(mt * 16 + half * 8 + g, c * 64 + q * 16) for g, q in lanes] for mt in range(step // 16) for half in range(2)
           for c in range(d // 64)], 16)
    check([[(kg * 16 + (t >> 1) * 8 + (t & 1) + 2 * q, g * (d // 8)) for g, q in lanes] for kg in range(step // 16)
           for t in range(4)], d // 8)
    # the rows in which a lane looks for NaN codes are those it reads
    for q in range(4):
        rows, row = [], 2 * q
        while row < step:
            rows.append(row)
            row += 7 if row & 1 else 1
        assert rows == sorted(kg * 16 + (t >> 1) * 8 + (t & 1) + 2 * q for kg in range(step // 16) for t in range(4))


@pytest.mark.parametrize("d,n_pairs", [(64, 32), (128, 64), (128, 32), (64, 8)])
def test_lanes_cover_each_channel_once_half(d, n_pairs):
    """The rotation's two vectors of a thread with the "half" pairing, pairs beside passing channels."""
    hit = np.zeros(d, int)
    for i in range(d // 16):
        half = n_pairs // 8
        a = 8 * i if i < half else 2 * n_pairs + 16 * (i - half)
        b = a + n_pairs if i < half else a + 8
        hit[a: a + 8] += 1
        hit[b: b + 8] += 1
    assert (hit == 1).all()


def test_plain_rounding_is_torch_e4m3():
    import torch
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-14, 9, 20000), [448, 449, 1e9, 0, -0.0],
                        np.arange(-64, 65) * 2.0 ** -10])
    got = torch.tensor(np.clip(x, -448, 448), dtype=torch.float64).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.round_e4m3(x.astype(np.float32).astype(np.float64)), got)
    assert np.array_equal(ref.VALUES[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())


def test_plain_rotation_gradient_by_differences():
    """The inverse rotation is the gradient: d(sum g . y)/dx by central differences."""
    rng = np.random.default_rng(5)
    for pairing in ("interleaved", "half"):
        x, g = rng.standard_normal((2, 3, 16))
        pos = rng.integers(0, 50, (3, 2))
        f, a = np.array([1.0, 0.3, 0.1, 0.7, 0.2, 0.05, 1.1, 0.6]), np.array([0, 1] * 4)
        got = ref.turn(g, pos, f, a, pairing, -1.0)
        for i in range(3):
            for c in range(16):
                e = np.zeros_like(x)
                e[i, c] = 1e-6
                num = ((ref.turn(x + e, pos, f, a, pairing) - ref.turn(x - e, pos, f, a, pairing)) * g).sum() / 2e-6
                assert abs(num - got[i, c]) < 1e-8

