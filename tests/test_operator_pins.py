"""CPU checks of what the operator tests lean on: the oracle's 4-bit codes,
rotation, score cap and distance bias against facts fixed outside it, the
workloads' 4-bit packing against the oracle's, and refusals that need no device."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_15_gb300 import binding as B
from paged_kv_cache_15_gb300 import build as pkv_build
from paged_kv_cache_15_gb300.workloads import (alibi_slopes, bf16_bits, fp4_pack_rows, make_workload, new_positions,
                                               rope_table)
from tests._operators import pool_values, reference


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return B.lib()


def test_e2m1_table_and_ties():
    assert oracle.e2m1_decode_array(np.arange(8)).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert oracle.e2m1_decode_array(np.arange(8, 16)).tolist() == [0, -0.5, -1, -1.5, -2, -3, -4, -6]
    for code in range(16):
        v = float(oracle.e2m1_decode_array([code])[0])
        assert int(oracle.e2m1_encode_array([v if code != 8 else -0.0])[0]) == code
    # every midpoint goes to the even code; beyond 6 saturates
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6, 7.0: 7, math.inf: 7}
    for x, code in ties.items():
        assert int(oracle.e2m1_encode_array([x])[0]) == code
        assert int(oracle.e2m1_encode_array([-x])[0]) == code + 8


@pytest.mark.parametrize("scale", [1.0, 1e-4, 3e4])
def test_fp4_packing_is_the_oracles(scale):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 3, 64, generator=g) * scale
    x[0, 0, :16] = 0.0
    x[1, 1, :16] = 1e-30
    x[2, 2, 5] = 1e30
    codes, scales = fp4_pack_rows(x, 0.7)
    ref_codes, ref_scales = oracle.fp4_encode_rows(x.numpy(), 0.7)
    assert np.array_equal(codes.numpy(), ref_codes) and np.array_equal(scales.numpy(), ref_scales)


def test_fp4_error_is_bounded_by_the_formats():
    """|x - code * S| <= max(half a step of the largest interval, saturation): with S within 2^-4 of max|x| / 6 (half a
    step of E4M3), every |z| <= 6 (1 + 2^-4), so the error is at most S (half of the step 2)."""
    x = np.random.default_rng(0).normal(size=(64, 2, 128)).astype(np.float32)
    codes, s8 = oracle.fp4_encode_rows(x, 1.0)
    s = np.repeat(oracle.e4m3_decode_array(s8), 16, axis=-1)
    assert (np.abs(oracle.e2m1_decode_array(codes) * s - x) <= s * (1 + 1e-6)).all()


def test_fp4_tiles_round_trip():
    rng = np.random.default_rng(1)
    pool = np.zeros(2 * 3 * 16 * 72, dtype=np.uint8)
    codes = rng.integers(0, 16, (32, 3, 128)).astype(np.uint8)
    scales = rng.integers(1, 0x7E, (32, 3, 8)).astype(np.uint8)
    loc = rng.permutation(32)
    oracle.fp4_store(pool, 3, loc, codes, scales)
    got = oracle.fp4_unpack(pool, 3, 128)
    want = oracle.e2m1_decode_array(codes) * np.repeat(oracle.e4m3_decode_array(scales), 16, -1)
    assert np.array_equal(got[loc], want)
    # the documented address of one code: slot 21, head 2, column 37
    i = int(np.argwhere(loc == 21)[0, 0])
    byte = pool[((21 // 16) * 3 + 2) * 1152 + (21 % 16) * 64 + 37 // 2]
    assert (byte >> 4) == codes[i, 2, 37]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(5, 2, 64)).astype(np.float32)
    table = rope_table(100, 32)
    pos = np.array([0, 1, 7, 99, 50])
    y = oracle.rotate(x, pos, table, 16, interleaved, np.float64)
    part = x[..., 16:48].astype(np.float64)
    z = part[..., 0::2] + 1j * part[..., 1::2] if interleaved else part[..., :16] + 1j * part[..., 16:]
    w = z * (table[pos, :16].astype(np.float64) + 1j * table[pos, 16:].astype(np.float64))[:, None]
    got = y[..., 16:48]
    re, im = (got[..., 0::2], got[..., 1::2]) if interleaved else (got[..., :16], got[..., 16:])
    assert np.abs(re - w.real).max() < 1e-14 and np.abs(im - w.imag).max() < 1e-14
    assert np.array_equal(y[..., :16], x[..., :16]) and np.array_equal(y[..., 48:], x[..., 48:])
    assert np.array_equal(y[0], x[0].astype(np.float64))  # position 0 turns nothing
    # the definition in fp32: three roundings, each at most half a step
    y32 = oracle.rotate(x, pos, table, 16, interleaved)
    assert np.abs(y32 - y).max() <= 3 * 2.0 ** -24 * 2 * np.abs(x).max()


@pytest.mark.parametrize("kv", ["bf16", "fp4_e2m1"])
def test_capped_and_biased_attention_against_loops(kv):
    """Brute force over keys on a tiny batch: c * tanh(s / c) + slope * (j - i), softmax, values."""
    W = make_workload("b", "extend", 2, 4, 2, 128, [3, 0], [2, 5], kv_dtype=kv)
    W.logit_cap, W.slopes = 2.0, alibi_slopes(4)
    from tests._operators import pools_after_append
    kp, vp = pools_after_append(W)
    k, v = pool_values(W, kp, 128) * W.k_scale, pool_values(W, vp, 128) * W.v_scale
    o, lse, _, _ = reference(W)
    q = W.q.double().numpy()
    t = 0
    for b in range(2):
        for i in range(int(W.qo_lens[b])):
            pos = int(W.prefix_lens[b]) + i
            for h in range(4):
                s, vals = [], []
                for j in range(pos + 1):
                    slot = int(W.page_table[b, j // 16]) * 16 + j % 16
                    x = float(q[t, h] @ k[slot, h // 2]) * W.sm_scale
                    s.append(2.0 * math.tanh(x / 2.0) + float(W.slopes[h]) * (j - pos))
                    vals.append(v[slot, h // 2])
                e = np.exp(np.array(s))
                assert abs(math.log(e.sum()) - lse[t, h]) < 1e-12
                assert np.abs((e[:, None] * np.array(vals)).sum(0) / e.sum() - o[t, h]).max() < 1e-12
            t += 1


def test_cap_and_bias_limits():
    """An endless cap and slopes of zero change nothing; a row's bias is 0 on its own key."""
    W = make_workload("l", "decode", 3, 4, 2, 64, [0, 20, 5], [1, 1, 1])
    plain = reference(W)
    W.logit_cap, W.slopes = 1e9, np.zeros(4, np.float32)
    same = reference(W)
    assert np.abs(plain[0] - same[0]).max() < 1e-12 and np.abs(plain[1] - same[1]).max() < 1e-12
    W.logit_cap, W.slopes = 0.0, alibi_slopes(4)
    biased = reference(W)
    assert np.allclose(biased[1][0], plain[1][0], atol=1e-12)  # one key: distance 0


def test_new_positions():
    assert new_positions([3, 0], [2, 3]).tolist() == [3, 4, 0, 1, 2]


def test_null_contexts_refused(lib):
    L = B.lib()
    rope = B.pkv_rope(None, 1, 16, 0, 0)
    assert L.pkv_rope_set_kv_buffer(None, ctypes.byref(rope), None, None, None, None, None, 0, None, 0, None, 0, None,
                                    1, 1.0, 1.0, None) == B.PKV_ERR_INVALID_ARG
    assert L.pkv_get_kv_buffer(None, None, None, None, None, None, 1, 1.0, 1.0, None) == B.PKV_ERR_INVALID_ARG
    assert L.pkv_set_logit_cap(None, 1.0) == B.PKV_ERR_INVALID_ARG
    assert L.pkv_set_alibi_slopes(None, None) == B.PKV_ERR_INVALID_ARG


def test_binding_checks_shapes_before_pointers():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    loc = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(4, 64)
    args = dict(loc=loc, positions=loc, cos_sin=table, q=t(2, 4, 64), k=t(2, 2, 64), v=t(2, 2, 64), q_out=t(2, 4, 64))
    for bad in (dict(positions=loc[:1]), dict(k=t(3, 2, 64)), dict(q_out=None), dict(q_out=t(2, 4, 32)),
                dict(cos_sin=table.double()), dict(cos_sin=table[0])):
        with pytest.raises(ValueError):
            B.pkv_rope_set_kv_buffer(None, t(1), t(1), **{**args, **bad})
    with pytest.raises(ValueError):
        B.pkv_get_kv_buffer(None, t(1), t(1), loc, t(2, 2, 64, dtype=torch.float32), t(2, 2, 64))
    with pytest.raises(ValueError):
        B.pkv_set_alibi_slopes(None, torch.zeros(4, dtype=torch.float64))


def test_fp4_pool_bytes_and_config(lib):
    cfg = B.make_config(32, 8, 128, 16, B.PKV_KV_FP4_E2M1, 10, 4, 100, 64)
    assert B.pkv_pool_bytes(cfg) == 10 * 8 * 1152
    n = ctypes.c_size_t(0)
    for kw, status in ((dict(head_dim=64), B.PKV_ERR_UNSUPPORTED), (dict(head_dim=192, head_dim_v=128),
                                                                     B.PKV_ERR_UNSUPPORTED)):
        args = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, kv_dtype=B.PKV_KV_FP4_E2M1,
                    num_pages=10, max_batch=4, max_pages_total=100, max_q_tokens=64)
        assert B.lib().pkv_workspace_bytes(ctypes.byref(B.make_config(**{**args, **kw})), ctypes.byref(n)) == status
    with pytest.raises(B.PkvError):  # slots that are not whole 16-slot tiles
        B.pkv_pool_bytes(B.make_config(32, 8, 128, 1, B.PKV_KV_FP4_E2M1, 10, 1, 1, 1))


def test_bf16_helpers_agree():
    x = torch.randn(64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    bits = bf16_bits(x)
    assert np.array_equal((bits.astype(np.uint32) << 16).view(np.float32), x.float().numpy())
