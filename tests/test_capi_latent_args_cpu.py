"""CPU checks of arguments of the latent cache's calls that the C entries and the binding refuse
before they touch a GPU."""
import ctypes

import pytest
import torch

from long_context_speculative_gb300 import build as lib_build
from long_context_speculative_gb300 import rapid

P = ctypes.c_void_p(256)        # a fake, aligned device address (never dereferenced)
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return rapid.lib()


def _z(*s, dtype=BF16):
    return torch.zeros(s, dtype=dtype)


def test_prefill_refuses_other_numbers_of_dimensions(lib):
    one = _z(1, dtype=I32)
    good = [_z(1, 3, 2, 192), _z(1, 9, 2, 128), _z(1, 9, 2, 128), _z(1, 9, 64)]
    for i in range(2):
        for bad in (good[i][0], good[i][None], _z(), good[i].flatten()):
            args = list(good)
            args[i] = bad
            with pytest.raises(rapid.RapidError):
                rapid.latent_prefill_attn(*args, one)
    with pytest.raises(rapid.RapidError):
        rapid.rapid_latent_prefill_attn(*good, one, None, 0.0, _z(1, 3, 2, 128), _z(1, 2, 3, dtype=torch.float32), None)


def test_read_refuses_other_numbers_of_dimensions_and_rows(lib):
    for cache, n in ((_z(), 3), (_z(64, 576), 3), (_z(1, 1, 64, 576), 3), (_z(1, 64, 576), 0), (_z(1, 64, 576), -1)):
        with pytest.raises(rapid.RapidError):
            rapid.latent_read(cache, None, n)


def test_append_refuses_query_rows_that_repeat(lib):
    # kv kv_strides q q_strides B n H weight eps inv flags prefix row_offset n_rows q_out cache type cap stream
    def call(strides, B=2, n=11, H=16):
        s = (ctypes.c_int64 * 6)(*strides)
        return lib.rapid_latent_append(P, None, P, s, B, n, H, P, ctypes.c_float(1e-6), P, 0, P, P, P, P, P, 1,
                                       4096, None)

    packed = [11 * 1024, 1024, 64]
    for i in range(3):
        for bad in (0, 8, 56):
            out = list(packed)
            out[i] = bad
            assert call(packed + out) == -1, (i, bad)


def test_commit_refuses_caches_that_overlap(lib):
    # caches layers type B cap n_q prefix path n_accepted stream
    size = {1: 2 * 64 * 1152, 2: 2 * 64 * 656}
    for code, nbytes in size.items():
        for at in ((0, 0), (0, nbytes - 16), (nbytes, 0, 2 * nbytes - 16), (3 * nbytes, 0, 5 * nbytes, 3 * nbytes)):
            table = (ctypes.c_void_p * len(at))(*[4096 + a for a in at])
            assert lib.rapid_latent_commit(table, len(at), code, 2, 64, 11, P, P, P, None) == -1, (code, at)
