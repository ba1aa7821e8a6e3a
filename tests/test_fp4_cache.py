"""Attention over 4-bit pools on every path against 64 bits: the step as a user
runs it (append by pkv_set_kv_buffer or with rotation, metadata, forward), so
codes written by the library are the ones its attention reads. Slots that hold
no token have NaN block scales."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_15_gb300 import binding as B
from paged_kv_cache_15_gb300.runner import DeviceBatch, config_for
from paged_kv_cache_15_gb300.workloads import (make_workload, new_positions, random_sinks, random_tree_masks,
                                               rope_table)
from tests._operators import check, pools_after_append, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_15_gb300 import build
    build.build()
    oracle.build()


def fp4(name, mode, bs, hq, hkv, prefix, new, page=16, rope=False, **kw):
    W = make_workload(name, mode, bs, hq, hkv, 128, prefix, new, page_size=page, kv_dtype="fp4_e2m1", **kw)
    if rope:
        W.cos_sin, W.positions = rope_table(int(W.seq_lens.max()), 128), new_positions(W.prefix_lens, W.qo_lens)
    return W


def run(W, spec=B.PKV_SPEC_PREFILL, cfg=None):
    d = DeviceBatch(W, cfg=cfg)
    d.step(spec)
    torch.cuda.synchronize()
    assert d.device_error() == 0
    return d


@pytest.mark.parametrize("page", [16, 128])
def test_append_bits(page):
    d = DeviceBatch(fp4("a", "extend", 5, 16, 8, [0, 40, 7, 100, 3], [37, 16, 1, 200, 90], page))
    d.set_kv_buffer()
    assert d.device_error() == 0
    for got, want in zip((d.k_pool, d.v_pool), pools_after_append(d.W)):
        assert np.array_equal(got.cpu().numpy(), want)


DECODE = {
    # query heads, KV heads, cached tokens: groups of 1 to 16 rows, lengths that end anywhere in a 16-slot tile, a
    # 128-key stage and a split
    "one_key": (8, 2, [0, 0, 0]),
    "tile_edges": (8, 2, [14, 15, 16, 17, 30, 31, 126, 127, 128, 129]),
    "mha": (4, 4, [5, 300, 77]),
    "g3": (6, 2, [1, 900, 450, 129]),
    "g4": (32, 8, [1023, 2, 511, 4000, 640]),
    "g8": (32, 4, [640, 63, 1500]),
    "g12": (36, 3, [700, 31, 2049]),
    "g16": (32, 2, [129, 2500, 16]),
    "long": (8, 1, [40000, 7]),
}


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("case", DECODE)
def test_decode(case, page):
    hq, hkv, cached = DECODE[case]
    check(run(fp4(case, "decode", len(cached), hq, hkv, cached, np.ones(len(cached)), page, rope=case != "long")))


def test_decode_padding_and_empty_batch():
    W = fp4("p", "decode", 4, 8, 2, [50, 20, 300, 9], np.ones(4))
    d = DeviceBatch(W)
    d.set_kv_buffer()
    W.seq_lens[[1, 3]] = 0
    d.seq_lens = torch.from_numpy(W.seq_lens).cuda()
    d.build_metadata()
    d.forward()
    torch.cuda.synchronize()
    assert d.device_error() == 0
    assert (d.out[[1, 3]] == 0).all() and torch.isneginf(d.lse[[1, 3]]).all()
    check(d)


@pytest.mark.parametrize("case", ["q2", "q4", "tc_rows128", "tc_one_row", "tc_ragged"])
@pytest.mark.parametrize("spec", ["prefill", "decode"])
def test_verify(case, spec):
    cfg = None
    if case == "q2":
        W = fp4(case, "verify", 4, 16, 4, [100, 0, 900, 15], [2, 1, 2, 2])
    elif case == "q4":
        W = fp4(case, "verify", 3, 8, 2, [1000, 33, 127], [4, 3, 1], rope=True)
    elif case == "tc_rows128":
        W = fp4(case, "verify", 4, 32, 4, [2500, 17, 900, 5100], [16, 16, 9, 16])
    elif case == "tc_one_row":
        W = fp4(case, "verify", 4, 64, 4, [2000, 300, 0, 129], np.ones(4))
        cfg = config_for(W, max_qo_len=8)
    else:
        W = fp4(case, "verify", 5, 64, 4, [2045, 126, 4380, 1999, 257], [4, 8, 5, 7, 6], page=128)
    check(run(W, B.PKV_SPEC_DECODE if spec == "decode" else B.PKV_SPEC_PREFILL, cfg))


EXTEND = {
    "one_token": (8, 2, [0], [1]),
    "ragged": (32, 8, [0, 37, 200, 15, 1023], [130, 9, 61, 1, 257]),
    "no_prefix": (8, 8, [0, 0, 0], [128, 129, 300]),
    "long_prefix": (16, 2, [3500, 127], [40, 300]),
    "g3": (6, 2, [16, 100], [200, 90]),
    "mixed_rows": (32, 4, [900, 64, 3000, 5], [1, 300, 2, 64]),
}


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("case", EXTEND)
def test_extend(case, page):
    hq, hkv, cached, new = EXTEND[case]
    check(run(fp4(case, "extend", len(cached), hq, hkv, cached, new, page, rope=case == "ragged")))


@pytest.mark.parametrize("spec", ["prefill", "decode"])
@pytest.mark.parametrize("what", ["tree", "sinks", "tree_and_sinks"])
def test_trees_and_sinks(what, spec):
    rng = np.random.default_rng(7)
    W = fp4("t", "verify", 4, 32, 4, rng.integers(0, 1500, 4), rng.integers(1, 13, 4))
    if "tree" in what:
        W.tree_mask = random_tree_masks(W.qo_lens, seed=8)
    if "sinks" in what:
        W.sinks = random_sinks(W.num_q_heads, seed=9)
    check(run(W, B.PKV_SPEC_DECODE if spec == "decode" else B.PKV_SPEC_PREFILL))


def test_decode_sinks():
    W = fp4("s", "decode", 3, 32, 8, [0, 700, 90], np.ones(3))
    W.sinks = random_sinks(32)
    check(run(W))


@pytest.mark.parametrize("mode", ["decode", "extend"])
def test_graph_replay_with_new_lengths(mode):
    """The whole step (append with rotation, metadata, forward) captured once and replayed with other lengths."""
    new = [1, 1, 1, 1] if mode == "decode" else [60, 1, 17, 129]
    W = fp4("g", mode, 4, 8, 2, [300, 40, 129, 77], new, rope=True)
    d = DeviceBatch(W)
    d.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.step()
    W2 = fp4("g", mode, 4, 8, 2, [200, 90, 16, 5], new, rope=True, num_pages=W.num_pages)
    d.W = W2
    for name, src in (("k_pool", W2.k_pool), ("v_pool", W2.v_pool), ("q", W2.q), ("k_new", W2.k_new),
                      ("v_new", W2.v_new), ("loc", torch.from_numpy(W2.loc)), ("seq_lens", torch.from_numpy(W2.seq_lens)),
                      ("positions", torch.from_numpy(W2.positions))):
        getattr(d, name).copy_(src)
    d.page_table[:, :W2.page_table.shape[1]].copy_(torch.from_numpy(W2.page_table))
    # pool scales are launch arguments: the new rows keep the captured ones
    W2.k_scale, W2.v_scale = W.k_scale, W.v_scale
    g.replay()
    torch.cuda.synchronize()
    assert d.device_error() == 0
    check(d)


def test_two_contexts_on_two_streams():
    ds = [DeviceBatch(fp4("c", "decode", 8, 32, 8, lens, np.ones(8)))
          for lens in (np.arange(8) * 211 + 5, np.arange(8)[::-1] * 317)]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(3):
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                d.step()
    torch.cuda.synchronize()
    for d in ds:
        assert d.device_error() == 0
        check(d)


def test_static_decode_is_the_context_decode():
    d = run(fp4("st", "decode", 3, 8, 2, [3, 400, 1000], np.ones(3)))
    out, lse = torch.full_like(d.out, 3.0), torch.full_like(d.lse, 3.0)
    err = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    W = d.W
    B.pkv_forward_decode_static(d.cfg, W.bs, d.seq_lens, d.page_table, d.q, d.k_pool, d.v_pool, W.sm_scale, out, lse,
                                err, W.k_scale, W.v_scale)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, d.out) and torch.equal(lse, d.lse)
    with pytest.raises(B.PkvError):
        B.pkv_forward_decode_static(d.cfg, W.bs, d.seq_lens, d.page_table, d.q, d.k_pool, d.v_pool, W.sm_scale, out,
                                    lse, err, 0.0, W.v_scale)


@pytest.mark.parametrize("case", ["decode", "extend", "verify_tc"])
def test_wait_limit_then_the_same_context_works(case):
    """A load that never comes makes the waits run out; afterwards the context works as before."""
    if case == "decode":
        W, spec = fp4("w", "decode", 3, 8, 2, [300, 20, 900], np.ones(3)), B.PKV_SPEC_PREFILL
    elif case == "extend":
        W, spec = fp4("w", "extend", 2, 8, 2, [300, 20], [150, 7]), B.PKV_SPEC_PREFILL
    else:
        W, spec = fp4("w", "verify", 2, 64, 4, [700, 20], [8, 3]), B.PKV_SPEC_DECODE
    d = DeviceBatch(W)
    B.pkv_set_wait_limit(d.ctx, 200_000)
    B.pkv_test_hold_first_load(d.ctx, True)
    d.step(spec)
    torch.cuda.synchronize()
    assert d.device_error() == B.PKV_DEV_TIMEOUT
    B.pkv_test_hold_first_load(d.ctx, False)
    B.pkv_set_wait_limit(d.ctx, 0)
    d.step(spec)
    torch.cuda.synchronize()
    assert d.device_error() == 0
    check(d)


@pytest.mark.parametrize("rows", [1, 40])
def test_results_do_not_change_between_runs(rows):
    W = fp4("d", "decode" if rows == 1 else "extend", 6, 32, 8, np.arange(6) * 700, np.full(6, rows))
    d = run(W)
    first = d.out.clone(), d.lse.clone()
    for _ in range(3):
        d.step()
    torch.cuda.synchronize()
    assert torch.equal(first[0], d.out) and torch.equal(first[1], d.lse)


def test_bad_page_recorded():
    W = fp4("b", "decode", 3, 8, 2, [100, 30, 60], np.ones(3))
    W.page_table[1, 1] = W.num_pages + 2
    d = DeviceBatch(W)
    d.build_metadata()
    d.forward()
    assert d.device_error() == B.PKV_DEV_BAD_PAGE


def test_non_positive_scales_rejected():
    d = run(fp4("n", "decode", 1, 8, 2, [10], [1]))
    for ks, vs in ((0.0, 1.0), (1.0, -1.0), (float("nan"), 1.0)):
        with pytest.raises(B.PkvError):
            B.pkv_forward(d.ctx, d.mode, 0, d.q, d.k_pool, d.v_pool, 1.0, d.out, d.lse, ks, vs)


def test_full_decode_batch():
    """64 requests of 1,024 to 8,192 keys, 32/8 heads: rows of three requests against 64 bits, and no NaN anywhere."""
    rng = np.random.default_rng(5)
    W = fp4("full", "decode", 64, 32, 8, rng.integers(1023, 8192, 64), np.ones(64))
    d = run(W)
    assert torch.isfinite(d.out.float()).all()
    for b in (0, 31, 63):
        Wb = fp4("one", "decode", 1, 32, 8, [int(W.prefix_lens[b])], [1])
        Wb.k_pool, Wb.v_pool, Wb.num_pages = W.k_pool, W.v_pool, W.num_pages
        Wb.page_table, Wb.seq_lens = W.page_table[b:b + 1], W.seq_lens[b:b + 1]
        Wb.q, Wb.k_new, Wb.v_new, Wb.loc = W.q[b:b + 1], W.k_new[b:b + 1], W.v_new[b:b + 1], W.loc[b:b + 1]
        Wb.k_scale, Wb.v_scale = W.k_scale, W.v_scale
        o, lse, tol, ltol = reference(Wb)
        assert (np.abs(d.out[b:b + 1].double().cpu().numpy() - o) <= tol).all()
        assert (np.abs(d.lse[b:b + 1].double().cpu().numpy() - lse) <= ltol).all()
