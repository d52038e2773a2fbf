"""What the token operators refuse beyond a single bad argument: tensors that overlap.  Nothing here reaches the GPU:
every call returns before a launch."""
import ctypes
import os

import pytest

from coo_spmm_fwd_amd import binding as csp

P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(csp.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return csp.load()


def test_grad_clip_refuses_tensors_that_overlap(lib):
    """One workgroup would read what another has scaled: the result would depend on which came first."""
    need = lib.grad_clip_workspace(3)
    dt = (ctypes.c_int32 * 3)(0, 0, 1)
    n = (ctypes.c_int64 * 3)(100, 50, 10)
    ptr = lambda *a: (ctypes.c_void_p * 3)(*a)

    def clip(g, o, n=n):
        return lib.grad_clip(g, o, n, dt, 3, ctypes.c_float(1.0), P, P, need, None)

    apart = ptr(4096, 8192, 12288)
    for g in (ptr(4096, 4096, 12288),      # one tensor listed twice, in place
              ptr(4096, 4492, 12288),      # one that begins in the last element of another
              ptr(12288, 8192, 12270)):    # in any order
        assert clip(g, g) == -1 and "overlap" in csp.sparse_layer_last_error()
    for o in (ptr(20480, 20480, 28672),    # outputs on each other
              ptr(8192, 20480, 28672),     # an output on another tensor's gradient
              ptr(4100, 20480, 28672),     # an output beside its own gradient's start
              ptr(20480, 24576, 24596)):
        assert clip(apart, o) == -1 and "overlap" in csp.sparse_layer_last_error()


def test_linear_ce_refuses_what_no_launch_could_hold(lib):
    """A launch has fewer than 2^32 threads: 256 a token, 512 a tile of 256 x 256 of dX."""
    for dt in (0, 1):
        for backward in (0, 1):
            size = lambda N, V, D: lib.linear_ce_workspace(N, V, D, dt, backward)
            assert size(2**24 - 64, 100, 8) > 0 and size(2**24 - 63, 100, 8) == -1
            assert size(2**22, 100, 2**16) > 0 and size(2**22, 100, 2**18) == -1
    assert lib.linear_ce_fwd(P, P, P, 2**24 - 63, 100, 8, 1, P, P, P, P, 2**60, None) == -1


def test_one_gradient_alone_refuses_as_both_do(lib):
    need = lib.linear_ce_workspace(4, 5, 8, 0, 1)
    for f in (lib.linear_ce_bwd_input, lib.linear_ce_bwd_weight):
        call = lambda X=P, W=P, t=P, N=4, V=5, D=8, dt=0, lse=P, dmean=P, total=P, out=P, w=P, nb=need: f(
            X, W, t, N, V, D, dt, lse, dmean, total, out, w, nb, None)
        for bad in ({"X": None}, {"W": None}, {"t": None}, {"lse": None}, {"dmean": None}, {"total": None}, {"out": None},
                    {"w": None}, {"nb": need - 1}, {"N": -1}, {"V": 0}, {"D": 0}, {"out": ctypes.c_void_p(4098)},
                    {"t": ctypes.c_void_p(4100)}, {"w": ctypes.c_void_p(4104)}):
            assert call(**bad) == -1, bad
        assert call(dt=3) == -6


def test_lookup_gradient_refuses_what_no_launch_could_hold(lib):
    """2^24 workgroups of 8 rows a lane group: dE of 280 GB."""
    for dt, V, D in ((0, 2**31 - 2, 33), (1, 2**31 - 2, 68), (0, 2**20, 2**19)):
        assert lib.embed_bwd_workspace(10, V, D, dt) == -1
        assert lib.embed_bwd(P, P, 10, V, D, dt, 1.0, P, P, 2**60, None) == -1
    assert lib.embed_bwd_workspace(10, 2**31 - 2, 16, 0) > 0 and lib.embed_bwd_workspace(10, 2**18, 2**18, 0) > 0
