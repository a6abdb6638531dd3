"""Refusals of spec_adjust_logits, and pins of its plain form (no GPU needed)."""
import ctypes
import os
import shutil

import numpy as np
import pytest

from oracle import paged


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from speculative_decoding_verification_53_gb300 import build
    build.build()
    import speculative_decoding_verification_53_gb300 as sv
    return sv.lib()


def test_arguments(lib):
    vp = ctypes.c_void_p(1 << 20)

    def call(logits=vp, dt=0, hist=None, hlen=None, H=0, bt=None, bv=None, M=0, B=1, R=3, V=100,
             out=ctypes.c_void_p(1 << 24)):
        return lib.spec_adjust_logits(logits, dt, hist, hlen, None, H, None, None, None, None, None, bt, bv, M, None,
                                      B, R, V, out, None)

    for bad in (dict(logits=None), dict(dt=2), dict(hist=vp, H=4), dict(H=-1), dict(H=2 ** 31 - 1), dict(M=-1),
                dict(M=65536), dict(bt=vp, M=2), dict(bv=vp, M=2), dict(B=-1), dict(B=65536), dict(R=0), dict(R=1026),
                dict(V=0), dict(V=(1 << 24) + 1), dict(out=None), dict(out=ctypes.c_void_p((1 << 20) + 4)),
                dict(logits=ctypes.c_void_p((1 << 20) + 2)), dict(out=ctypes.c_void_p((1 << 20) - 8))):
        assert call(**bad) == 1, bad
    assert call(B=0, logits=None, out=None) == 0


def test_plain_form_pins():
    """One token by hand: seen in the prompt, counted in output and drafts, biased, masked."""
    x = np.array([[[2.0, -2.0, 1.0, 0.5, 7.0]] * 3])
    got = paged.adjust_logits(x, history=np.array([[0, 1, 1]]), history_len=[3], prompt_len=[1],
                              draft_tokens=np.array([[1, 2]]), repetition=[2.0], presence=[0.5], frequency=[0.25],
                              bias_tokens=np.array([[3, 3, -1]]), bias_values=np.array([[9.0, 1.0, 4.0]]),
                              allowed=np.array([[[0b01111], [0b01111], [0]]], np.uint32))
    assert got[0, 0].tolist() == [1.0, -4 - 0.5 - 0.5, 1.0, 1.5, -np.inf]
    assert got[0, 1].tolist() == [1.0, -4 - 0.75 - 0.5, 1.0, 1.5, -np.inf]
    assert np.isneginf(got[0, 2]).all()
    tree = paged.adjust_logits(x, draft_tokens=np.array([[2, 2]]), tree_mask=np.array([[[1], [2]]], np.uint32),
                               frequency=[1.0])
    assert tree[0, :, 2].tolist() == [1.0, 0.0, 0.0]  # siblings do not count each other
