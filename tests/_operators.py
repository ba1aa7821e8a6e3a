"""What the operator tests share: pools as the oracle sees them after the append
(rotated where the workload says so), the attention of a workload with its
error bound, and bf16 helpers."""
import numpy as np
import torch

import oracle
from paged_kv_cache_15_gb300.workloads import Workload, bf16_bits
from tests._pipeline import oracle_meta


def bf16_to_f32(t: torch.Tensor) -> np.ndarray:
    return t.float().numpy()


def f32_to_bf16(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def rotated(W: Workload):
    """(q, k) of the step's tokens, fp32: rotated as the operator is defined, or as they are."""
    q, k = bf16_to_f32(W.q), bf16_to_f32(W.k_new)
    if W.cos_sin is None:
        return q, k
    turn = lambda x: oracle.rotate(x, W.positions, W.cos_sin, W.rotary_offset, W.interleaved)  # noqa: E731
    return turn(q), turn(k)


def pools_after_append(W: Workload, pools=None):
    """The pools' bytes after the step's append: numpy arrays of the pools' shapes."""
    _, k = rotated(W)
    v = bf16_to_f32(W.v_new)
    out = []
    for pool, x, inv in ((W.k_pool, k, W.k_inv_scale), (W.v_pool, v, W.v_inv_scale)):
        if W.is_fp4:
            p = pool.numpy().copy()
            oracle.fp4_store(p, W.num_kv_heads, W.loc, *oracle.fp4_encode_rows(x, inv))
        elif W.is_fp8:
            p = pool.numpy().copy()
            with np.errstate(all="ignore"):
                y = (x * np.float32(inv)).astype(np.float32)
            p[W.loc] = np.array([oracle.e4m3_encode(float(e)) for e in y.ravel()], dtype=np.uint8).reshape(y.shape)
        else:
            p = bf16_bits(pool).copy()
            p[W.loc] = bf16_bits(f32_to_bf16(x))
        out.append(p)
    return out


def pool_values(W: Workload, pool, width):
    """Decoded values [slots, heads, width] of a pool's bytes, without the pool's scale."""
    if W.is_fp4:
        return oracle.fp4_unpack(pool, W.num_kv_heads, width)
    if W.is_fp8:
        return oracle.e4m3_decode_array(pool)
    return (pool.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def reference(W: Workload):
    """(o, lse, bound of o's error, bound of lse's error) of every row in 64 bits.

    With A = sum_j w_j |v_j| of a row: the output's rounding is off by at most
    2^-8 |o|, the weights' (bf16 2^-8, f16 for coded pools 2^-11) by that times
    A, a split's partial rows by 2^-8 A, and the fp32 scores by under 5e-5
    each, which moves every weight and the normaliser by that share (1e-4 A).
    """
    kp, vp = pools_after_append(W)
    kv, vv = pool_values(W, kp, W.head_dim), pool_values(W, vp, W.dv)
    q, _ = rotated(W)
    qb = bf16_bits(f32_to_bf16(q))
    meta = oracle_meta(W)

    def attend(values):
        return oracle.attention(qb, kv, values, meta, W.num_q_heads, W.num_kv_heads, W.page_size, W.sm_scale,
                                kv_dtype=oracle.KV_F64, k_scale=W.k_scale, v_scale=W.v_scale, tree_mask=W.tree_mask,
                                sinks=None if W.sinks is None else W.sinks.astype(np.float64),
                                logit_cap=W.logit_cap, slopes=W.slopes)

    o, lse = attend(vv)
    a, _ = attend(np.abs(vv))
    weights = 2.0 ** -8 if W.kv_dtype == "bf16" else 2.0 ** -11
    tol = 2.0 ** -8 * np.abs(o) + (weights + 2.0 ** -8 + 1e-4) * a + 1e-30
    return o, lse, tol, 1e-4 + 1e-6 * np.abs(np.where(np.isfinite(lse), lse, 0.0))


def check(d, ref=None):
    """A DeviceBatch's outputs against the reference of its workload."""
    o, lse, tol, ltol = ref if ref is not None else reference(d.W)
    got, glse = d.out.double().cpu().numpy(), d.lse.double().cpu().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - o)
    assert (err <= tol).all(), f"o: {(err > tol).sum()} of {err.size}, worst {(err / tol).max():.3g} of the bound"
    none = np.isneginf(lse)
    assert np.array_equal(none, np.isneginf(glse))
    lerr = np.where(none, 0.0, np.abs(np.where(none, 0.0, glse) - np.where(none, 0.0, lse)))
    assert (lerr <= ltol).all(), f"lse: worst {(lerr / ltol).max():.3g} of the bound"
