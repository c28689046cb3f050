"""CPU checks of the 8-bit cache's C ABI and binding: bad host-side arguments are refused
before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

from long_context_speculative_gb300 import build as lib_build
from long_context_speculative_gb300 import rapid

import _q8

P = ctypes.c_void_p(256)        # a fake, aligned device address (never dereferenced)
ODD = ctypes.c_void_p(264)      # 8-byte aligned only
BYTE = ctypes.c_void_p(257)


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return rapid.lib()


def _refused(call, good, changes, status=-1):
    for i, bad in changes:
        args = list(good)
        args[i] = bad
        assert call(*args) == status, (i, bad)


def test_qkv_append(lib):
    f = ctypes.c_float
    # q k v strides dtype B n Hq Hkv d qw kw eps inv rot flags prefix pos row n_rows Q K V cap stream
    good = [P, P, P, None, 1, 2, 11, 32, 8, 128, P, P, f(1e-6), P, 128, 0, P, P, P, P, P, P, P, 4096, None]
    _refused(lib.rapid_qkv_append, good,
             [(0, None), (1, None), (2, None), (4, 2), (5, 0), (6, 0), (7, 0), (8, 0), (9, 96),
              (12, f(-1.0)), (12, f(float("nan"))), (12, f(float("inf"))), (13, None), (14, 8),
              (14, 144), (14, -16), (15, 2), (16, None), (20, None), (21, None), (22, None), (23, 0),
              (0, ODD), (1, ODD), (2, ODD), (10, ODD), (11, ODD), (20, ODD), (21, ODD), (22, ODD),
              (13, BYTE), (16, BYTE), (17, BYTE), (18, BYTE), (19, BYTE), (7, 65536)])
    for i in range(6):
        for bad in (4, -8):       # 8 bytes of bf16; negative
            s = [4096] * 6
            s[i] = bad
            args = list(good)
            args[3] = (ctypes.c_int64 * 6)(*s)
            assert lib.rapid_qkv_append(*args) == -1, (i, bad)


def _seal_args():
    arr = (ctypes.c_void_p * 1)(256)
    # K V pages scales layers dtype B Hkv d cap keep n_pages table max_pages sealed tail stream
    return [arr, arr, arr, arr, 1, 1, 2, 8, 128, 256, 0, 10, P, 5, P, P, None]


def test_kv_seal(lib):
    _refused(lib.rapid_kv_seal, _seal_args(),
             [(0, None), (1, None), (2, None), (3, None), (4, 0), (4, 129), (5, 3), (6, 0), (7, 0),
              (7, 40000), (8, 96), (9, 0), (10, -1), (11, 0), (12, None), (13, 0), (13, (1 << 24) + 1),
              (14, None), (15, None), (12, BYTE), (14, BYTE), (15, BYTE),
              (0, (ctypes.c_void_p * 1)(264)), (2, (ctypes.c_void_p * 1)(264)),
              (3, (ctypes.c_void_p * 1)(258)), (1, (ctypes.c_void_p * 1)(None))])
    good = [P, P, P, 2, 5, 10, 256, 0, None]
    _refused(lib.rapid_kv_seal_advance, good,
             [(0, None), (1, None), (2, None), (3, 0), (4, 0), (5, 0), (6, 0), (7, -1), (0, BYTE)])


def test_verify_attn_q8(lib):
    f = ctypes.c_float
    size = lib.rapid_verify_attn_q8_workspace_size
    need = size(1, 32, 8, 128, 11, 256, 100, 1)
    assert need > 0
    for i, bad in [(0, 0), (1, 0), (1, 30), (2, 0), (3, 96), (4, 0), (4, 65), (5, 10), (6, 0),
                   (6, (1 << 24) + 1), (7, 2)]:
        args = [1, 32, 8, 128, 11, 256, 100, 1]
        args[i] = bad
        assert size(*args) == 0, (i, bad)
    assert size(8192, 8, 8, 128, 5, 64, 10, 1) == 0              # B * Hkv
    assert size(1, 128, 1, 128, 64, 64, 10, 1) == 0              # group rows
    # Q K V pages scales table dtype B Hq Hkv d n_q cap n_pages max_pages sealed tail mask scale O LSE ws
    good = [P, P, P, P, P, P, 1, 1, 32, 8, 128, 11, 256, 100, 100, P, P, None, f(0.0), P, P, P, need, None]
    _refused(lib.rapid_verify_attn_q8, good,
             [(0, None), (1, None), (2, None), (3, None), (4, None), (5, None), (15, None), (16, None),
              (19, None), (20, None), (21, None), (6, 2), (7, 0), (10, 32), (11, 0), (11, 65), (12, 10),
              (13, 0), (13, 1 << 22), (14, 0), (0, ODD), (1, ODD), (2, ODD), (3, ODD), (19, ODD),
              (21, ODD), (4, ctypes.c_void_p(260)), (5, BYTE), (15, BYTE), (16, BYTE), (20, BYTE),
              (18, f(float("inf"))), (18, f(float("nan")))])
    _refused(lib.rapid_verify_attn_q8, good, [(22, need - 1)], status=-3)


def test_verify_attn_q8_counts_key_tiles_in_32_bits(lib):
    size = lib.rapid_verify_attn_q8_workspace_size
    assert size(120, 8, 8, 128, 1, 64, 1 << 24, 1) > 0
    assert size(128, 8, 8, 128, 1, 64, 1 << 24, 1) == 0          # 128 * 2^24 page tiles and more
    assert size(64, 8, 8, 128, 1, 1 << 31, 100, 1) == 0 and size(63, 8, 8, 128, 1, 1 << 31, 100, 1) > 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    c = _q8.cache(1, 2, 128, torch.bfloat16, [2], [5], 3, seed=1)
    Q = torch.zeros((1, 4, 3, 128), dtype=torch.bfloat16)
    with pytest.raises(rapid.RapidError):
        rapid.verify_attn_q8(Q, c["K"], c["V"], c["pages"], c["scales"], c["page_table"],
                             c["sealed_len"], c["tail_len"])
    with pytest.raises(rapid.RapidError):
        rapid.Q8LayerTable([c["K"]], [c["V"]], [c["pages"]], [c["scales"]])
    with pytest.raises(rapid.RapidError):
        rapid.Q8LayerTable([], [], [], [])
    rows = torch.zeros((1, 3, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(rapid.RapidError):
        rapid.qkv_append(rows, rows[:, :, :2], rows[:, :, :2], c["K"], c["V"], c["tail_len"])


# ---------------------------------------------------------------------------
# The 64-bit forms that the GPU tests compare with
# ---------------------------------------------------------------------------

def test_reference_rounding_is_e4m3():
    x = np.concatenate([np.linspace(-448, 448, 4001), np.linspace(-0.05, 0.05, 4001),
                        [2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 1.1875, 240.0, 464.0 - 16]])
    got = torch.tensor(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(_q8.e4m3_round(x), got)


def test_reference_scale():
    assert _q8.block_scale(448.0) == 1.0 and _q8.block_scale(448.1) == 2.0
    assert _q8.block_scale(0.0) == 1.0 and _q8.block_scale(1e-30) == 2.0 ** -64
    assert _q8.block_scale(3.0) == 2.0 ** -7


def test_reference_attention_by_hand():
    # two keys of one page with values 1 and 3, one tail row with value 5: equal scores
    pages = torch.zeros((1, 1, 2, 64, 64)).to(torch.float8_e4m3fn)
    scales = torch.ones((1, 1, 2))
    pages[0, 0, 1] = torch.ones((64, 64)).to(torch.float8_e4m3fn)
    scales[0, 0, 1] = 2.0
    K = torch.zeros((1, 1, 16, 64))
    V = torch.full((1, 1, 16, 64), 5.0)
    Q = torch.zeros((1, 1, 1, 64))
    one = torch.ones(1, dtype=torch.int32)
    O, L, _, _ = _q8.attn(Q, K, V, pages, scales, torch.zeros((1, 1), dtype=torch.int32), 64 * one, 0 * one)
    assert torch.allclose(O, torch.full_like(O, (64 * 2 + 5) / 65), rtol=1e-14)
    assert abs(float(L) - np.log(65)) < 1e-12


def test_reference_rotation_by_hand():
    # position 3 at one radian per position; norm of (3, 4, 0, ...) is 5 / 8
    q = torch.zeros((1, 1, 1, 64))
    q[..., 0], q[..., 32] = 3.0, 4.0
    K = torch.zeros((1, 1, 16, 64))
    inv = torch.zeros(32)
    inv[0] = 1.0
    w = torch.full((64,), 2.0)
    Q, K2, V2, _, _ = _q8.append(q, q, q, K, K, torch.zeros((1, 1, 1, 64)), torch.tensor([3]), inv, w, None,
                                 eps=0.0)
    a, b = 3 / (5 / 8) * 2, 4 / (5 / 8) * 2
    c, s = np.cos(3.0), np.sin(3.0)
    assert abs(float(Q[0, 0, 0, 0]) - (a * c - b * s)) < 1e-12
    assert abs(float(Q[0, 0, 0, 32]) - (b * c + a * s)) < 1e-12
    assert abs(float(K2[0, 0, 3, 0]) - (3 * c - 4 * s)) < 1e-12
    assert float(V2[0, 0, 3, 32]) == 4.0 and float(K2.abs().sum()) > 0
