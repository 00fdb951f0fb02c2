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
])
def test_rope_refuses(lib, change, rc):
    assert lib.fvattn_rope(*rope_args(**change)) == rc


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
    (dict(ws_bytes=64), CAPACITY), (dict(M=100, ws_bytes=64, os=strides(0, 6400, 64)), CAPACITY),
])
def test_attend_refuses(lib, change, rc):
    assert lib.fvattn_cache_attend(*attend_args(**change)) == rc


def test_attend_workspace(lib):
    import top_routed_block_b200 as fv
    ws = fv.fvattn_cache_attend_workspace_bytes
    assert ws(0, 1, 1, 1, 64, 64, 1) == 0 and ws(1, 1, 1, 1, 96, 64, 1) == 0 and ws(4097, 1, 1, 1, 64, 64, 1) == 0
    # more than 32 rows: K and V of every page as bf16
    assert ws(2, 3, 4, 9, 128, 128, 5) >= 2 * 2 * 3 * 5 * 128 * 128 * 2
    # few rows: bounded by the grid, not by the cache's length
    assert 0 < ws(1, 8, 1, 1, 128, 128, 1 << 20) < 64 << 20
    assert ws(1, 1, 1, 1, 64, 64, 1) <= 4096 + 8 * 68 * 4


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
    // the plan: whole steps, every token once, no more items than the workspace has room for
    std::srand(7);
    for (int it = 0; it < 20000; ++it) {
        const int B = 1 + std::rand() % 20, step = 128;
        const long groups = 1 + std::rand() % 90, ctas = 1 + std::rand() % 443;
        const long cap = 64L * (1 + std::rand() % (it % 3 ? 60 : 20000));
        std::vector<long> len(B);
        long tokens = 0, items = 0;
        for (long &x : len) {
            x = std::rand() % 4 ? std::rand() % (cap + 1) : 0;
            tokens += x > 0 ? x : 1;
        }
        const long chunk = chunk_tokens(tokens, groups, ctas, 4, step);
        CHECK(chunk >= step && chunk % step == 0);
        for (long x : len) {
            const long n = chunks_of(x, chunk);
            CHECK(n >= 1 && n * chunk >= x && (n - 1) * chunk < (x > 0 ? x : 1));
            items += n * groups;
        }
        CHECK(items <= max_items(B, groups, cap, ctas, 4, step));
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


@pytest.mark.parametrize("d", [64, 128])
def test_lanes_cover_each_cached_byte_once(d):
    """The few-rows kernel's loads of a step of 32 tokens: every byte of the 32 rows by one lane."""
    for kind in ("k", "v"):
        hit = np.zeros(32 * d, int)
        for lane in range(32):
            g, q = lane >> 2, lane & 3
            if kind == "k":
                at = [g * d + q * 16 + (mt * 16 + hf * 8) * d + c * 64 for mt in range(2) for hf in range(2)
                      for c in range(d // 64)]
                size = 16
            else:
                at = [g * (d // 8) + 2 * q * d + (kg * 16 + (t >> 1) * 8 + (t & 1)) * d for kg in range(2)
                      for t in range(4)]
                size = d // 8
            for a in at:
                assert a % size == 0
                hit[a: a + size] += 1
        assert (hit == 1).all()


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

