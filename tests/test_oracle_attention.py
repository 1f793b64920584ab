"""Pins of the attention oracle and of the host arithmetic of the rotary frequencies (no GPU)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import attention as ref


@pytest.fixture(scope="module")
def mlora():
    from rank_adapter_gemm_token_gb300 import build, mlora
    build.build()
    mlora.load()
    return mlora


def test_one_key_returns_its_value():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(1, 2, 4)), rng.normal(size=(1, 1, 4)), rng.normal(size=(1, 1, 4))
    out, _, _ = ref.attention(q, [k], [v], [0, 1], 2, 0.5)
    assert np.array_equal(out, np.repeat(v, 2, 1))


def test_hand_worked_two_keys():
    # scores ln 3 and 0: weights 3/4 and 1/4
    q = np.array([[[1.0, 0.0]]])
    k = np.array([[[math.log(3.0), 5.0]], [[0.0, -7.0]]])
    v = np.array([[[4.0, 8.0]], [[0.0, 16.0]]])
    out, _, _ = ref.attention(q, [k], [v], [0, 1], 1, 1.0)
    assert np.allclose(out, [[[3.0, 10.0]]], rtol=1e-14)


def test_causal_rows_equal_shorter_sequences():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(5, 2, 4)), rng.normal(size=(9, 2, 4)), rng.normal(size=(9, 2, 4))
    out, _, _ = ref.attention(q, [k], [v], [0, 5], 1, 0.3)
    for t in range(5):
        one, _, _ = ref.attention(q[t:t + 1], [k[:5 + t]], [v[:5 + t]], [0, 1], 1, 0.3)
        assert np.allclose(out[t], one[0], rtol=1e-14)


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(2)
    freq = [1.0, 0.1, 0.01]
    x, y = rng.normal(size=(2, 1, 1, 8))
    for inter in (False, True):
        a = ref.rotate(x, np.array([70]), freq, inter)
        assert np.isclose(np.linalg.norm(a), np.linalg.norm(x))
        assert np.array_equal(a[..., 6:], x[..., 6:])
        near = (ref.rotate(x, np.array([3]), freq, inter) * ref.rotate(y, np.array([5]), freq, inter)).sum()
        far = (ref.rotate(x, np.array([103]), freq, inter) * ref.rotate(y, np.array([105]), freq, inter)).sum()
        assert np.isclose(near, far)


def test_e4m3_values():
    v = ref.e4m3_values()
    assert v[1] == 2.0 ** -9 and v[7] == 7 * 2.0 ** -9 and v[8] == 2.0 ** -6 and v[126] == 448.0 and v[56] == 1.0


def test_rope_frequencies(mlora):
    rot, theta = 64, 10000.0
    plain = np.array(mlora.mlora_rope_frequencies(rot, theta))
    assert np.allclose(plain, theta ** (-2.0 * np.arange(32) / rot), rtol=1e-14)
    linear = np.array(mlora.mlora_rope_frequencies(rot, theta, mlora.MLORA_ROPE_LINEAR, 4.0))
    assert np.allclose(linear, plain / 4, rtol=1e-14)
    base = np.array(mlora.mlora_rope_frequencies(rot, theta, mlora.MLORA_ROPE_BASE, 4.0))
    assert base[0] == 1.0 and np.isclose(base[-1], plain[-1] / 4, rtol=1e-12) and np.all(np.diff(base / plain) < 0)
    waves = np.array(mlora.mlora_rope_frequencies(rot, theta, mlora.MLORA_ROPE_WAVES, 8.0, 4096.0, 1.0, 4.0))
    turns = 4096 * plain / (2 * math.pi)
    assert np.allclose(waves[turns >= 4], plain[turns >= 4]) and np.allclose(waves[turns <= 1], plain[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 4)
    share = (turns[mid] - 1) / 3
    assert mid.any() and np.allclose(waves[mid], plain[mid] * (share + (1 - share) / 8), rtol=1e-12)
    ramp = np.array(mlora.mlora_rope_frequencies(rot, theta, mlora.MLORA_ROPE_RAMP, 8.0, 4096.0, 1.0, 32.0))
    pair = lambda n: rot * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = math.floor(pair(32.0)), math.ceil(pair(1.0))
    i = np.arange(32)
    share = 1 - np.clip((i - lo) / (hi - lo), 0, 1)
    assert np.allclose(ramp, plain * (share + (1 - share) / 8), rtol=1e-12)


@pytest.mark.parametrize("args", [(0, 1e4, 0, 1, 0, 0, 0), (7, 1e4, 0, 1, 0, 0, 0), (64, 1.0, 0, 1, 0, 0, 0),
                                  (64, float("nan"), 0, 1, 0, 0, 0), (64, 1e4, 5, 1, 0, 0, 0), (64, 1e4, 1, 0.5, 0, 0, 0),
                                  (2, 1e4, 2, 2, 0, 0, 0), (64, 1e4, 3, 2, 0, 1, 4), (64, 1e4, 4, 2, 4096, 4, 1)])
def test_rope_frequencies_refuse(mlora, args):
    with pytest.raises(mlora.MloraError) as e:
        mlora.mlora_rope_frequencies(*args)
    assert e.value.status == mlora.MLORA_ERR_INVALID_ARG


def test_refusals_need_no_device(mlora):
    lib, bad, out = mlora.load(), mlora.MLORA_ERR_INVALID_ARG, ctypes.c_void_p()
    create = lambda *a: lib.mlora_kv_create(*a, None, None, None, None, ctypes.byref(out))  # noqa: E731
    for sizes in ((0, 16, 8, 128, 0), (4, 12, 8, 128, 0), (4, 4, 8, 128, 0), (4, 512, 8, 128, 0), (4, 16, 0, 128, 0),
                  (4, 16, 257, 128, 0), (4, 16, 8, 96, 0), (4, 16, 8, 128, 2), (1 << 24, 256, 1, 64, 0)):
        assert create(*sizes) == bad and not out.value, sizes
    assert lib.mlora_kv_create(4, 16, 8, 128, 0, None, None, None, None, None) == bad
    assert lib.mlora_kv_create(4, 16, 8, 128, 0, 256, None, None, None, ctypes.byref(out)) == bad       # K without V
    assert lib.mlora_kv_create(4, 16, 8, 128, 1, 256, 256, None, None, ctypes.byref(out)) == bad        # e4m3 without scales
    assert lib.mlora_kv_create(4, 16, 8, 128, 0, 256, 256, 256, 256, ctypes.byref(out)) == bad          # bf16 with scales
    assert lib.mlora_kv_create(4, 16, 8, 128, 0, 264, 256, None, None, ctypes.byref(out)) == bad        # misaligned
    for sizes in ((0, 4, 4, 8, 8, 128), (8193, 4, 4, 8, 8, 128), (4, 0, 4, 8, 8, 128), (4, 65536, 4, 8, 8, 128),
                  (4, 4, 0, 8, 8, 128), (8192, 4, 1 << 18, 8, 8, 128), (4, 4, 4, 8, 3, 128), (4, 4, 4, 4, 8, 128),
                  (4, 4, 4, 8, 8, 80), (4, 4, 4, 512, 8, 128)):
        assert lib.mlora_seq_create(*sizes, ctypes.byref(out)) == bad, sizes
    freq = (ctypes.c_double * 64)(*[1.0] * 64)
    for rot in (0, 4, 12, 136):
        assert lib.mlora_rope_create(rot, 0, freq, 1.0, ctypes.byref(out)) == bad
    assert lib.mlora_rope_create(64, 0, None, 1.0, ctypes.byref(out)) == bad
    assert lib.mlora_rope_create(64, 0, freq, float("inf"), ctypes.byref(out)) == bad
    freq[3] = float("nan")
    assert lib.mlora_rope_create(64, 0, freq, 1.0, ctypes.byref(out)) == bad
    for call in (lib.mlora_build_seq(None, None, None, None, 1, 0, 0, 0, None, None), lib.mlora_seq_status(None),
                 lib.mlora_qkv_write(None, None, None, 0, None, None, 0.0, None, None, None, None),
                 lib.mlora_attention(None, None, None, 1.0, None, None), lib.mlora_kv_read(None, None, None, 0, None, None, None),
                 lib.mlora_kv_info(None, *[None] * 9)):
        assert call == bad
    assert lib.mlora_kv_destroy(None) == 0 and lib.mlora_seq_destroy(None) == 0 and lib.mlora_rope_destroy(None) == 0
    assert mlora.mlora_kv_bytes(10, 16, 8, 128, 0) == 2 * 10 * 16 * 8 * 128 * 2
    assert mlora.mlora_kv_bytes(10, 16, 8, 128, 1) == 2 * 10 * 16 * 8 * (128 + 4)
    assert mlora.mlora_kv_bytes(10, 17, 8, 128, 1) == 0
