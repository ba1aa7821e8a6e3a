"""pkv_rope_set_kv_buffer and pkv_get_kv_buffer on the GPU: every stored bit
against the operator's definition (fp32, each product and sum rounded once),
the rotated queries against the formula in 64 bits, and what the calls refuse,
skip and leave alone."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_15_gb300 import binding as B
from paged_kv_cache_15_gb300.runner import KV_OF
from paged_kv_cache_15_gb300.workloads import fp4_pool, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_15_gb300 import build
    build.build()
    oracle.build()


class Step:
    """n tokens' q, k, v as slices of fused rows, and pools of `pages` pages with known old bytes."""

    def __init__(self, n, hq, hkv, dk, dv, kv, rot, first=0, inter=False, page=16, seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.n, self.hq, self.hkv, self.dk, self.dv, self.kv = n, hq, hkv, dk, dv, kv
        self.first, self.inter = first, inter
        pages = -(-(n + 40) // page) + 1
        slots = pages * page
        x = torch.from_numpy(rng.normal(size=(n, hq * dk + hkv * (dk + dv) + 8)).astype(np.float32) * spread)
        self.fused = x.to(torch.bfloat16).cuda()
        self.q = self.fused[:, :hq * dk].view(n, hq, dk)
        self.k = self.fused[:, hq * dk:(hq + hkv) * dk].view(n, hkv, dk)
        self.v = self.fused[:, (hq + hkv) * dk:-8].view(n, hkv, dv)
        self.loc = torch.from_numpy(rng.permutation(slots)[:n].astype(np.int32)).cuda()
        self.table = rope_table(5000, rot)
        self.pos = rng.integers(0, 5000, n).astype(np.int32)
        self.q_out = torch.full((n, hq, dk), 7.0, dtype=torch.bfloat16, device="cuda")
        self.inv = (1.7, 0.9) if kv != "bf16" else (1.0, 1.0)
        if kv == "fp4_e2m1":  # y of N(0, 1) input near the scale range's middle
            self.inv = (170.0, 90.0)
        self.old = []
        for d in (dk, dv):
            if kv == "bf16":
                self.old.append(torch.from_numpy(rng.integers(0, 1 << 15, (slots, hkv, d)).astype(np.int16)))
            elif kv == "fp8_e4m3":
                self.old.append(torch.from_numpy(rng.integers(0, 256, (slots, hkv, d)).astype(np.uint8)))
            else:
                self.old.append(fp4_pool(slots, hkv, d))
        self.pools = [p.cuda() for p in self.old]
        if kv == "bf16":
            self.pools = [p.view(torch.bfloat16) for p in self.pools]
        self.attn = B.PagedAttention(B.make_config(hq, hkv, dk, page, KV_OF[kv], pages, 1, 1, 1, 1,
                                                   head_dim_v=dv if dv != dk else 0))
        self.ctx = self.attn.ctx
        self.cos_sin, self.positions = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.pos).cuda()

    def call(self, **kw):
        args = dict(loc=self.loc, positions=self.positions, cos_sin=self.cos_sin, q=self.q, k=self.k, v=self.v,
                    q_out=self.q_out, rotary_offset=self.first, interleaved=self.inter, k_inv_scale=self.inv[0],
                    v_inv_scale=self.inv[1])
        args.update(kw)
        B.pkv_rope_set_kv_buffer(self.ctx, *self.pools, **args)

    def turned(self, x, dtype=np.float32):
        return oracle.rotate(x.float().cpu().numpy(), self.positions.cpu().numpy(), self.table, self.first, self.inter,
                             dtype)

    def expected_pools(self, keep=None):
        """Old bytes with the new rows (of the tokens in `keep`) stored."""
        keep = np.arange(self.n) if keep is None else keep
        loc = self.loc.cpu().numpy()[keep]
        out = []
        for old, x, inv in zip(self.old, (self.turned(self.k), self.v.float().cpu().numpy()), self.inv):
            p, x = old.numpy().copy(), x[keep]
            with np.errstate(all="ignore"):
                y = (x * np.float32(inv)).astype(np.float32)
            if self.kv == "bf16":
                p[loc] = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy()
            elif self.kv == "fp8_e4m3":
                p[loc] = np.array([oracle.e4m3_encode(float(e)) for e in y.ravel()], dtype=np.uint8).reshape(y.shape)
            else:
                oracle.fp4_store(p, self.hkv, loc, *oracle.fp4_encode_rows(x, inv))
            out.append(p)
        return out

    def check_pools(self, keep=None):
        for got, want in zip(self.pools, self.expected_pools(keep)):
            g = got.view(torch.int16) if self.kv == "bf16" else got
            assert np.array_equal(g.cpu().numpy().reshape(want.shape), want)

    def error(self):
        return B.pkv_get_device_error(self.ctx)


SHAPES = [
    # n, hq, hkv, dk, dv, kv, rot, first, inter, page
    (1, 8, 2, 64, 64, "bf16", 64, 0, False, 16),
    (7, 8, 2, 64, 64, "bf16", 16, 48, True, 128),
    (33, 6, 3, 128, 128, "bf16", 96, 8, False, 16),     # half of 48: partner vectors off the 16-column grid
    (5, 6, 3, 192, 128, "bf16", 64, 128, True, 16),
    (19, 4, 1, 192, 128, "bf16", 192, 0, False, 128),
    (1, 32, 8, 128, 128, "fp8_e4m3", 128, 0, False, 16),
    (21, 8, 8, 128, 128, "fp8_e4m3", 48, 24, False, 16),
    (1, 8, 2, 128, 128, "fp4_e2m1", 128, 0, False, 16),
    (37, 6, 3, 128, 128, "fp4_e2m1", 48, 24, False, 128),
    (50, 32, 4, 128, 128, "fp4_e2m1", 64, 64, True, 16),
    (1400, 32, 8, 128, 128, "bf16", 128, 0, False, 16),  # four heads a thread
    (2001, 30, 2, 128, 128, "fp8_e4m3", 128, 0, True, 16),  # and head counts that four does not divide
    (1800, 30, 6, 128, 128, "fp4_e2m1", 128, 0, False, 128),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[5]}-n{s[0]}-{s[1]}x{s[2]}x{s[3]}-r{s[6]}+{s[7]}")
def test_stored_bits_and_queries(shape):
    n, hq, hkv, dk, dv, kv, rot, first, inter, page = shape
    s = Step(n, hq, hkv, dk, dv, kv, rot, first, inter, page)
    s.call()
    assert s.error() == 0
    s.check_pools()
    q = torch.from_numpy(s.turned(s.q)).to(torch.bfloat16)
    assert torch.equal(s.q_out.cpu().view(torch.int16), q.view(torch.int16))
    # and against the formula in 64 bits: one bf16 rounding, three fp32 ones of terms up to |a| + |b|
    y = s.turned(s.q, np.float64)
    size = np.abs(s.q.float().cpu().numpy()).max()
    assert (np.abs(s.q_out.double().cpu().numpy() - y) <= 2.0 ** -8 * np.abs(y) + 3 * 2.0 ** -24 * 2 * size).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "fp4_e2m1"])
def test_contiguous_inputs_and_no_queries(kv):
    s = Step(9, 8, 2, 128, 128, kv, 128)
    s.k, s.v = s.k.contiguous(), s.v.contiguous()
    s.call(q=None, q_out=None)
    assert s.error() == 0
    s.check_pools()
    assert (s.q_out == 7.0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "fp4_e2m1"])
def test_bad_slots_and_positions_skip_their_token(kv):
    s = Step(12, 8, 2, 128, 128, kv, 64)
    s.loc[3] = -1
    s.loc[5] = 1 << 30
    s.call()
    assert s.error() == B.PKV_DEV_BAD_SLOT
    good = np.array([i for i in range(12) if i not in (3, 5)])
    s.check_pools(good)
    assert torch.equal(s.q_out.cpu(), torch.from_numpy(s.turned(s.q)).to(torch.bfloat16))  # their queries turn
    t = Step(12, 8, 2, 128, 128, kv, 64)
    keep_pos = t.positions.clone()
    t.positions[0] = 5000
    t.positions[11] = -7
    t.call()
    assert t.error() == B.PKV_DEV_BAD_POSITION
    t.positions.copy_(keep_pos)
    good = np.arange(1, 11)
    t.check_pools(good)
    assert (t.q_out[[0, 11]] == 7.0).all() and not (t.q_out[1:11] == 7.0).all()


@pytest.mark.parametrize("kv", ["fp8_e4m3", "fp4_e2m1"])
def test_saturation_infinities_and_nan(kv):
    s = Step(6, 8, 2, 128, 128, kv, 32, 96, spread=1e6)
    s.k[0, 0, 3] = float("inf")   # not rotated
    s.k[1, 1, 17] = float("nan")
    s.v[2, 0, 0] = float("-inf")
    s.v[3, 1, 127] = float("nan")
    s.v[4] = 0.0
    s.call()
    assert s.error() == 0
    if kv == "fp8_e4m3":
        s.check_pools()
        return
    for got, want in zip(s.pools, s.expected_pools()):
        # codes of a block whose scale is NaN may be anything: the values are what counts
        a, b = (oracle.fp4_unpack(p, 2, 128) for p in (got.cpu().numpy(), want))
        assert np.array_equal(a, b, equal_nan=True)


def test_bf16_pools_keep_unrotated_bits():
    s = Step(4, 8, 2, 128, 128, "bf16", 64)
    s.fused.view(torch.int16)[:, 8 * 128 + 64: 8 * 128 + 72] = 0x7FA5  # NaNs with payloads, columns 64.. of k head 0
    s.v.view(torch.int16)[0, 0, :4] = 0x7F81
    s.call()
    assert (s.pools[0].view(torch.int16)[s.loc.long(), 0, 64:72] == 0x7FA5).all()
    assert (s.pools[1].view(torch.int16)[s.loc.long()[0], 0, :4] == 0x7F81).all()


def test_no_tokens_is_a_no_op():
    s = Step(3, 8, 2, 64, 64, "bf16", 64)
    e = lambda t: t[:0]  # noqa: E731
    s.call(loc=e(s.loc), positions=e(s.positions), q=e(s.q), k=e(s.k), v=e(s.v), q_out=e(s.q_out))
    assert s.error() == 0
    s.check_pools(np.zeros(0, dtype=int))


def test_capture_and_replay_with_new_positions_on_another_stream():
    s = Step(16, 8, 2, 128, 128, "fp4_e2m1", 128)
    s.call()
    torch.cuda.synchronize()
    g, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=stream):
        s.call()
    for p, old in zip(s.pools, s.old):
        p.copy_(old)
    s.positions.copy_(torch.arange(16, dtype=torch.int32) * 31)
    s.loc.copy_(s.loc.flip(0))
    s.q_out.zero_()
    with torch.cuda.stream(stream):
        stream.wait_stream(torch.cuda.default_stream())
        g.replay()
    stream.synchronize()
    assert s.error() == 0
    s.check_pools()
    assert torch.equal(s.q_out.cpu(), torch.from_numpy(s.turned(s.q)).to(torch.bfloat16))


def test_refusals_launch_nothing():
    s = Step(4, 8, 2, 128, 128, "fp8_e4m3", 64)

    def refused(**kw):
        with pytest.raises(B.PkvError) as e:
            s.call(**kw)
        assert e.value.status == B.PKV_ERR_INVALID_ARG

    refused(rotary_offset=72)                        # 72 + 64 > 128
    refused(rotary_offset=-8)
    refused(rotary_offset=4)                         # not a multiple of 8
    refused(cos_sin=torch.zeros(10, 24, device="cuda"))  # rotary_dim 24
    refused(cos_sin=torch.zeros(0, 64, device="cuda"))
    refused(k_inv_scale=0.0)
    refused(v_inv_scale=float("inf"))
    refused(k_inv_scale=float("nan"))
    big = torch.zeros(4, 8 * 128 + 4, dtype=torch.bfloat16, device="cuda")
    refused(q=big[:, :8 * 128].view(4, 8, 128))      # token stride not a multiple of 8
    refused(q=s.q_out, q_out=s.q_out)                # in place: other threads still read their partner columns
    flat = torch.zeros(4 * 8 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    refused(q_out=flat[1:1 + 4 * 8 * 128].view(4, 8, 128))  # misaligned
    with pytest.raises(ValueError):
        s.call(loc=s.loc.long())
    with pytest.raises(ValueError):
        s.call(q=s.q.transpose(1, 2).contiguous().transpose(1, 2))
    assert s.error() == 0
    s.check_pools(np.zeros(0, dtype=int))
    assert (s.q_out == 7.0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "fp4_e2m1"])
@pytest.mark.parametrize("n", [1, 45])
def test_read_back(kv, n):
    s = Step(n, 8, 3 if kv != "bf16" else 2, 192 if kv == "bf16" else 128, 128, kv, 64) if kv == "bf16" else Step(
        n, 6, 3, 128, 128, kv, 64)
    s.call()
    loc = torch.cat([s.loc, s.loc[:1]])  # a slot may repeat
    k = torch.full((n + 1, s.hkv, s.dk), 5.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full((n + 1, s.hkv, s.dv), 5.0, dtype=torch.bfloat16, device="cuda")
    scales = (0.0123, 3.7)
    B.pkv_get_kv_buffer(s.ctx, *s.pools, loc, k, v, *scales)
    assert s.error() == 0
    for got, pool, scale, d in zip((k, v), s.expected_pools(), scales, (s.dk, s.dv)):
        if kv == "bf16":
            want = torch.from_numpy(pool[loc.cpu().numpy()])
            assert torch.equal(got.view(torch.int16).cpu(), want)
            continue
        values = oracle.fp4_unpack(pool, s.hkv, d) if kv == "fp4_e2m1" else oracle.e4m3_decode_array(pool)
        want = (values[loc.cpu().numpy()].astype(np.float32) * np.float32(scale)).astype(np.float32)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))
    loc[0] = -1
    k.fill_(5.0)
    B.pkv_get_kv_buffer(s.ctx, *s.pools, loc, k, v, *scales)
    assert s.error() == B.PKV_DEV_BAD_SLOT
    assert (k[0] == 5.0).all() and not (k[-1] == 5.0).all()
    if kv != "bf16":
        with pytest.raises(B.PkvError):
            B.pkv_get_kv_buffer(s.ctx, *s.pools, loc, k, v, 0.0, 1.0)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "fp4_e2m1"])
def test_slots_past_two_gigabytes(kv):
    """Element offsets of a pool's last slots pass 32 bits (E4M3) and its byte offsets 31 bits (4-bit)."""
    hkv, pages = 8, (1 << 18) + 16  # 4.2 M slots of 1,024 elements
    attn = B.PagedAttention(B.make_config(8, hkv, 128, 16, KV_OF[kv], pages, 1, 1, 1, 1))
    nbytes = B.pkv_pool_bytes(B.make_config(8, hkv, 128, 16, KV_OF[kv], pages, 1, 1, 1, 1))
    pools = [torch.zeros(nbytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.randn(3, hkv, 128, generator=g, device="cuda").bfloat16()
    loc = torch.tensor([pages * 16 - 1, 0, pages * 16 - 40], dtype=torch.int32, device="cuda")
    table = torch.from_numpy(rope_table(4, 128)).cuda()
    B.pkv_rope_set_kv_buffer(attn.ctx, *pools, loc, torch.zeros_like(loc), table, None, x, x, None, k_inv_scale=32.0,
                             v_inv_scale=32.0)
    k, v = torch.zeros_like(x), torch.zeros_like(x)
    B.pkv_get_kv_buffer(attn.ctx, *pools, loc, k, v, 1 / 32, 1 / 32)
    assert B.pkv_get_device_error(attn.ctx) == 0
    assert torch.equal(k, v)  # position 0 turns nothing
    # E4M3 is off by half a step, 2^-4; 4-bit codes by a block's scale (max / 6, within 2^-4)
    tol = 2.0 ** -4 * x.abs().float() + 2.0 ** -8 if kv == "fp8_e4m3" else (
        x.float().unflatten(-1, (8, 16)).abs().amax(-1, keepdim=True) / 6 * (1 + 2.0 ** -3)).expand(3, hkv, 8, 16).flatten(-2)
    assert ((k.float() - x.float()).abs() <= tol).all()
