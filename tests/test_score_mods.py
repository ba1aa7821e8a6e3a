"""Score cap and distance bias on every path and pool type against 64 bits, the
limits in which they change nothing, and what is refused."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_15_gb300 import binding as B
from paged_kv_cache_15_gb300.runner import DeviceBatch
from paged_kv_cache_15_gb300.workloads import (alibi_slopes, make_workload, new_positions, random_sinks,
                                               random_tree_masks, rope_table)
from tests._operators import check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_15_gb300 import build
    build.build()
    oracle.build()


CASES = {
    # mode, spec, query heads, KV heads, K width, V width, cached, new
    "decode_g4": ("decode", 0, 32, 8, 128, 128, [0, 15, 700, 129, 1600], [1] * 5),
    "decode_g3_d64": ("decode", 0, 6, 2, 64, 64, [3, 64, 900], [1] * 3),
    "decode_g16": ("decode", 0, 32, 2, 128, 128, [77, 500, 1], [1] * 3),
    "decode_192": ("decode", 0, 8, 2, 192, 128, [30, 600], [1] * 2),
    "verify_rows16": ("verify", 1, 16, 4, 128, 128, [100, 0, 900], [4, 3, 1]),
    "verify_tc": ("verify", 1, 64, 4, 128, 128, [2045, 126, 300], [4, 8, 5]),
    "verify_prefill": ("verify", 0, 64, 4, 128, 128, [2045, 126, 300], [4, 8, 5]),
    "extend": ("extend", 0, 32, 8, 128, 128, [0, 37, 1023, 15], [130, 9, 300, 1]),
    "extend_g3_d64": ("extend", 0, 6, 2, 64, 64, [16, 0], [200, 90]),
    "extend_192": ("extend", 0, 8, 2, 192, 128, [30, 200], [77, 140]),
    "extend_long_prefix": ("extend", 0, 8, 1, 128, 128, [5000, 2], [20, 3]),
}


def work(case, kv="bf16", cap=0.0, slopes=False, page=16, gain=1.0):
    mode, spec, hq, hkv, dk, dv, cached, new = CASES[case]
    W = make_workload(case, mode, len(cached), hq, hkv, dk, cached, new, page_size=page, kv_dtype=kv,
                      head_dim_v=dv if dv != dk else None)
    W.q = (W.q.float() * gain).to(torch.bfloat16)
    W.logit_cap = cap
    W.slopes = alibi_slopes(hq) if slopes else None
    return W, spec


def run(W, spec):
    d = DeviceBatch(W)
    d.step(spec)
    torch.cuda.synchronize()
    assert d.device_error() == 0
    return d


@pytest.mark.parametrize("what", ["cap", "bias", "both"])
@pytest.mark.parametrize("case", CASES)
def test_bf16_pools(case, what):
    W, spec = work(case, cap=0.0 if what == "bias" else 5.0, slopes=what != "cap", gain=4.0)
    check(run(W, spec))


@pytest.mark.parametrize("kv", ["fp8_e4m3", "fp4_e2m1"])
@pytest.mark.parametrize("case", ["decode_g4", "decode_g16", "verify_tc", "verify_prefill", "extend"])
def test_coded_pools(case, kv):
    W, spec = work(case, kv=kv, cap=30.0, slopes=True, page=128, gain=3.0)
    W.sinks = random_sinks(W.num_q_heads)
    check(run(W, spec))


@pytest.mark.parametrize("case", ["decode_g4", "extend"])
@pytest.mark.parametrize("cap", [0.01, 1.0, 50.0, 1e4])
def test_caps_from_flat_to_none(case, cap):
    """A tiny cap makes every score nearly equal, a saturated one +-cap; an endless one changes nothing."""
    W, spec = work(case, cap=cap, gain=50.0 if cap < 1e4 else 1.0)
    if cap == 1e4:
        # the cap's rounding grows with it: 2^-22 * cap * log2(e) in the log2 domain
        ref = reference(W)
        d = run(W, spec)
        off = 4 * 2.0 ** -22 * cap
        a = ref[2] / (2.0 ** -7 + 1e-4)
        check(d, (ref[0], ref[1], ref[2] + 2 * off * a, ref[3] + off))
        return
    check(run(W, spec))


@pytest.mark.parametrize("case", ["decode_g4", "extend", "verify_tc"])
@pytest.mark.parametrize("cap", [1e-30, 1e-10, 1e20, 1e30])
def test_caps_at_the_ends_of_their_range(case, cap):
    """A vanishing cap leaves every visible key the same weight; a vast one leaves the scores alone, to their last bits."""
    W, spec = work(case, cap=cap)
    check(run(W, spec))


@pytest.mark.parametrize("case", ["decode_g16", "extend_g3_d64", "verify_prefill"])
def test_scores_on_both_sides_of_the_polynomial(case):
    """Scores up to several caps: the polynomial near zero and the quotient beyond it in the same rows."""
    W, spec = work(case, cap=2.0, gain=1.0)
    check(run(W, spec))
    W, spec = work(case, cap=1.7, gain=2.5, slopes=True)
    check(run(W, spec))


@pytest.mark.parametrize("case", ["decode_g4", "extend_long_prefix", "verify_tc"])
def test_steep_and_positive_and_zero_slopes(case):
    W, spec = work(case, slopes=True)
    W.slopes = np.linspace(0.0, 8.0, W.num_q_heads).astype(np.float32)  # one key is all a steep head sees
    check(run(W, spec))
    W.slopes = np.full(W.num_q_heads, -0.001, np.float32)  # far keys favoured
    check(run(W, spec))
    W.slopes = np.zeros(W.num_q_heads, np.float32)
    check(run(W, spec))


def test_padding_rows_stay_empty():
    W, spec = work("decode_g4", cap=20.0, slopes=True)
    d = DeviceBatch(W)
    d.set_kv_buffer()
    W.seq_lens[[1, 4]] = 0
    d.seq_lens = torch.from_numpy(W.seq_lens).cuda()
    d.build_metadata()
    d.forward()
    torch.cuda.synchronize()
    assert (d.out[[1, 4]] == 0).all() and torch.isneginf(d.lse[[1, 4]]).all()
    check(d)


def test_cap_with_trees_and_slopes_with_trees_refused():
    W, _ = work("verify_tc", cap=10.0)
    W.tree_mask = random_tree_masks(W.qo_lens)
    for spec in (0, 1):
        check(run(W, spec))
    W16, spec = work("verify_rows16", cap=10.0, gain=3.0)
    W16.tree_mask = random_tree_masks(W16.qo_lens)
    check(run(W16, spec))
    d = DeviceBatch(W)
    d.set_kv_buffer()
    d.build_metadata()
    d.out.fill_(7.0)
    slopes = torch.from_numpy(alibi_slopes(W.num_q_heads)).cuda()
    B.pkv_set_alibi_slopes(d.ctx, slopes)
    for spec in (0, 1):
        with pytest.raises(B.PkvError) as e:
            d.forward(spec)
        assert e.value.status == B.PKV_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert (d.out == 7.0).all()
    B.pkv_set_alibi_slopes(d.ctx, None)
    d.forward(1)
    torch.cuda.synchronize()
    check(d)


@pytest.mark.parametrize("case", ["decode_g4", "extend", "verify_tc"])
def test_off_again_gives_the_plain_results(case):
    W, spec = work(case)
    d = run(W, spec)
    plain = d.out.clone(), d.lse.clone()
    B.pkv_set_logit_cap(d.ctx, 3.0)
    slopes = torch.from_numpy(alibi_slopes(W.num_q_heads)).cuda()
    B.pkv_set_alibi_slopes(d.ctx, slopes)
    d.forward(spec)
    assert not torch.equal(plain[0], d.out)
    B.pkv_set_logit_cap(d.ctx, 0.0)
    B.pkv_set_alibi_slopes(d.ctx, None)
    d.forward(spec)
    torch.cuda.synchronize()
    assert torch.equal(plain[0], d.out) and torch.equal(plain[1], d.lse)


def test_refusals():
    W, _ = work("decode_g3_d64")
    d = DeviceBatch(W)
    for cap in (-1.0, float("nan"), float("inf"), 1e31, 1e-31):
        with pytest.raises(B.PkvError) as e:
            B.pkv_set_logit_cap(d.ctx, cap)
        assert e.value.status == B.PKV_ERR_INVALID_ARG
    raw = torch.zeros(64, dtype=torch.uint8, device="cuda")
    assert B.lib().pkv_set_alibi_slopes(d.ctx, raw.data_ptr() + 2) == B.PKV_ERR_INVALID_ARG
    d.step()
    torch.cuda.synchronize()
    check(d)


def test_whole_step_replayed_with_new_slopes():
    """Rotation with append, metadata and a capped, biased forward in one graph; the slopes are read at replay."""
    W, _ = work("extend", cap=8.0, slopes=True, gain=3.0)
    W.cos_sin, W.positions = rope_table(2000, 64), new_positions(W.prefix_lens, W.qo_lens)
    W.rotary_offset = 32
    d = DeviceBatch(W)
    d.step()
    torch.cuda.synchronize()
    check(d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.step()
    W.slopes = (alibi_slopes(W.num_q_heads)[::-1] * 0.3).copy()
    d.slopes.copy_(torch.from_numpy(W.slopes))
    d.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert d.device_error() == 0
    check(d)
