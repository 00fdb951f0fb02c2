"""What the entry points of the rotary positions and the cache refuse, each change by itself: the unchanged
arguments pass every check (outputs lie apart from inputs) and fail only where a GPU is looked for."""
import ctypes

import pytest
import torch

from tests.test_cache_cpu import (ALIGNMENT, CAPACITY, FAKE, INVALID, P, UNSUPPORTED, append_args, attend_args, freqs, lib,  # noqa: F401
                                  rope_args, strides)

OUT = P(1 << 20)
NO_GPU = (-5, -2)   # a CUDA error, or no supported device: behind the argument checks


def rope(lib, **kw):  # noqa: F811
    return lib.fvattn_rope(*rope_args(**{"Qr": OUT, **kw}))


def attend(lib, **kw):  # noqa: F811
    return lib.fvattn_cache_attend(*attend_args(**{"O": OUT, **kw}))


@pytest.mark.skipif(torch.cuda.is_available(), reason="would run")
def test_unchanged_arguments_pass(lib):  # noqa: F811
    for got in (rope(lib), attend(lib), lib.fvattn_cache_append(*append_args())):
        assert got in NO_GPU


@pytest.mark.parametrize("change,rc", [
    (dict(pos=None), INVALID), (dict(freq=None), INVALID), (dict(axis=None), INVALID), (dict(B=0), INVALID), (dict(N=0), INVALID),
    (dict(qh=0), INVALID), (dict(n_pairs=0), INVALID), (dict(n_pairs=33), INVALID), (dict(n_axes=0), INVALID),
    (dict(n_axes=5), UNSUPPORTED), (dict(pairing=2), INVALID), (dict(pairing=-1), INVALID), (dict(pairing=1, n_pairs=12), UNSUPPORTED),
    (dict(inverse=2), INVALID), (dict(kh=1), INVALID), (dict(K=FAKE), INVALID), (dict(Kr=FAKE), INVALID), (dict(pos_b=7), INVALID),
    (dict(qs=strides(0, -64, 64)), INVALID), (dict(qs=strides(-64, 64, 64)), INVALID), (dict(qs=strides(0, 64, 4)), ALIGNMENT),
    (dict(qs=None), INVALID), (dict(qrs=None), INVALID), (dict(qrs=strides(0, 0, 64)), INVALID),
    (dict(qrs=strides(0, 64, 64)), INVALID), (dict(qrs=strides(0, 640, 32)), INVALID), (dict(qrs=strides(0, 636, 64)), ALIGNMENT),
    (dict(B=2, qrs=strides(640, 640, 64)), INVALID), (dict(pos=P(18)), ALIGNMENT), (dict(Qr=P(18)), ALIGNMENT),
    (dict(Qr=FAKE), INVALID),   # where Q lies, with other strides
])
def test_rope(lib, change, rc):  # noqa: F811
    assert rope(lib, **change) == rc


@pytest.mark.parametrize("freq,axis", [(float("nan"), 0), (float("inf"), 0), (1.0, -1), (1.0, 1)])
def test_rope_pairs(lib, freq, axis):  # noqa: F811
    for i in (0, 17, 31):
        f, a = freqs(32)
        f[i], a[i] = freq, axis
        assert rope(lib, freq=f, axis=a) == INVALID


@pytest.mark.parametrize("change,rc", [
    (dict(LSE=None), INVALID), (dict(lens=None), INVALID), (dict(ws=None), INVALID), (dict(status=None), INVALID), (dict(Q=None), INVALID),
    (dict(O=None), INVALID), (dict(qs=None), INVALID), (dict(os=None), INVALID), (dict(table=None), INVALID), (dict(kc=None), INVALID),
    (dict(ke=None), INVALID), (dict(vc=None), INVALID), (dict(ve=None), INVALID), (dict(num_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(B=0), INVALID), (dict(heads=0), INVALID), (dict(M=0), INVALID), (dict(group=0), INVALID),
    (dict(causal=2), INVALID), (dict(causal=-1), INVALID), (dict(os=strides(0, 0, 64)), INVALID), (dict(M=3, os=strides(0, 64, 64)), INVALID),
    (dict(qs=strides(0, -64, 64)), INVALID), (dict(qs=strides(0, 3, 64)), ALIGNMENT), (dict(O=P(24)), ALIGNMENT),
    (dict(LSE=P(18)), ALIGNMENT), (dict(lens=P(18)), ALIGNMENT), (dict(new=P(18)), ALIGNMENT), (dict(ws=P(24)), ALIGNMENT),
    (dict(kc=P(24)), ALIGNMENT), (dict(ke=P(18)), ALIGNMENT), (dict(table=P(18)), ALIGNMENT), (dict(status=P(18)), ALIGNMENT),
    (dict(d=96), UNSUPPORTED), (dict(block=32), UNSUPPORTED), (dict(B=4097), UNSUPPORTED), (dict(max_pages=1 << 25), UNSUPPORTED),
    (dict(group=1 << 12, M=1 << 12), UNSUPPORTED), (dict(ws_bytes=64), CAPACITY),
    (dict(M=100, ws_bytes=64, os=strides(0, 6400, 64)), CAPACITY), (dict(O=FAKE), INVALID),   # where Q lies
])
def test_attend(lib, change, rc):  # noqa: F811
    assert attend(lib, **change) == rc


@pytest.mark.parametrize("change,rc", [
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(heads=0), INVALID), (dict(vs=strides(0, -64, 64)), INVALID),
    (dict(vs=strides(0, 64, 4)), ALIGNMENT), (dict(V=P(24)), ALIGNMENT), (dict(vc=P(24)), ALIGNMENT), (dict(start=P(18)), ALIGNMENT),
    (dict(new=P(18)), ALIGNMENT), (dict(status=P(18)), ALIGNMENT), (dict(pos=P(18)), ALIGNMENT), (dict(pos=FAKE, pairing=2), INVALID),
    (dict(pos=FAKE, freq=None), INVALID), (dict(pos=FAKE, axis=None), INVALID), (dict(pos=FAKE, n_axes=0), INVALID),
    (dict(pos=FAKE, n_axes=5), UNSUPPORTED), (dict(pos=FAKE, pairing=1, n_pairs=12), UNSUPPORTED), (dict(T=(1 << 31) - 1, heads=40), UNSUPPORTED),
])
def test_append(lib, change, rc):  # noqa: F811
    assert lib.fvattn_cache_append(*append_args(**change)) == rc
