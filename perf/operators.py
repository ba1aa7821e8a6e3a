"""Cases of the operators around the paged KV cache: what each computes in plain
torch operations, and the framework's calls for the same work.

Three families, told apart by a case's "op":

* "rope": one step's q, k and v, slices of a fused projection's rows, have q and
  k rotated by their positions and k and v appended to the paged pools (bf16,
  E4M3, or 4-bit codes with block scales; a 4-bit case reads the appended rows
  back, as a server does that moves cached prefixes).
* "fp4": attention over pools held in 4 bits (decode, extend, verify).
* "bias": attention whose scores are capped by a tanh and / or biased by the
  distance of query and key (decode, extend, verify).

A 4-bit pool holds, for every 16 slots and KV head, one tile: 16 rows of D/2
bytes (two E2M1 codes each, even column in the low nibble), then 16 rows of
D/16 E4M3 block scales; value = code * block scale * pool scale.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
E2M1_MAX = 6.0
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MAX_POSITIONS = 131072


# ---------------------------------------------------------------- the cases
def _rope(name, tokens, hq, hkv, dk, dv, rot, kv, first=0, inter=False, far=0, page=16):
    """first: first rotated column; far: positions start there."""
    case = dict(op="rope", tokens=tokens, hq=hq, hkv=hkv, dk=dk, dv=dv, rot=rot, first=first, inter=inter, kv=kv,
                far=far, page=page)
    return dict(case, name=name) if name else case


def _attn(name, op, mode, bs, hq, hkv, d, lo, hi, mix, n_lo=1, n_hi=1, kv="bf16", cap=0.0, alibi=False, page=16,
          empty=0, tc=False):
    """bs requests whose cached lengths lie in [lo, hi] and new tokens in [n_lo, n_hi] (drawn from mix), the
    first `empty` of them padding (no key at all); tc: verify on the decode path."""
    case = dict(op=op, mode=mode, bs=bs, hq=hq, hkv=hkv, d=d, lo=lo, hi=hi, mix=mix, n_lo=n_lo, n_hi=n_hi, kv=kv,
                cap=cap, alibi=alibi, page=page, empty=empty, tc=tc)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one decode step of four requests of a small model: latency
        _rope("rope_step_small", 4, 8, 2, 64, 64, 64, "bf16"),
        # one decode step of 64 requests with long contexts, E4M3 cache
        _rope("rope_step_64_e4m3", 64, 32, 8, 128, 128, 128, "e4m3", far=100000),
        # a full prefill batch
        _rope("rope_prefill_bf16", 16384, 32, 8, 128, 128, 128, "bf16"),
        # a ragged prefill batch into a 4-bit cache, and its rows read back
        _rope("rope_prefill_fp4", 8189, 32, 8, 128, 128, 128, "fp4"),
        # four short requests, one of them graph padding: latency
        _attn("fp4_decode_small", "fp4", "decode", 4, 8, 2, 128, 36, 299, 1, kv="fp4", empty=1),
        # an 8-billion-parameter model's decode batch
        _attn("fp4_decode_64", "fp4", "decode", 64, 32, 8, 128, 1023, 8191, 2, kv="fp4"),
        # long contexts, what a 4-bit cache is for
        _attn("fp4_decode_long", "fp4", "decode", 8, 32, 8, 128, 32767, 131071, 3, kv="fp4"),
        # prefill over a cached prefix
        _attn("fp4_extend", "fp4", "extend", 8, 32, 8, 128, 0, 4096, 4, n_lo=128, n_hi=2048, kv="fp4"),
        # short ragged requests with a distance bias
        _attn("bias_decode_short", "bias", "decode", 21, 32, 8, 128, 0, 300, 5, alibi=True, empty=2),
        # a decode batch of a model that caps its scores
        _attn("cap_decode_64", "bias", "decode", 64, 32, 8, 128, 1023, 8191, 6, cap=50.0),
        # prefill of a model that caps its scores
        _attn("cap_extend", "bias", "extend", 8, 32, 8, 128, 0, 4096, 7, n_lo=128, n_hi=2048, cap=50.0),
        # speculative drafts verified with both, E4M3 cache
        _attn("cap_bias_verify", "bias", "verify", 32, 64, 4, 128, 2048, 16384, 8, n_lo=4, n_hi=8, kv="e4m3", cap=30.0,
              alibi=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "fp4", "bias"))
    page = rng.choice((16, 128))
    if op == "rope":
        kv = rng.choice(("bf16", "e4m3", "fp4"))
        hq, hkv = rng.choice(((8, 2), (40, 8), (32, 4), (64, 4), (4, 4), (6, 3)))
        dk, dv = rng.choice(((64, 64), (128, 128), (192, 128))) if kv == "bf16" else (128, 128)
        rot = rng.choice([r for r in (16, 32, 64, 128, 192) if r <= dk])
        first = rng.choice((0, dk - rot))
        most = int(16384 * 32 * 128 / max(32 * 128, hq * dk))
        return _rope(None, _log_int(rng, 1, most), hq, hkv, dk, dv, rot, kv, first, rng.choice((False, True)),
                     rng.choice((0, 5, 40000, 110000)), page)
    mode = rng.choice(("decode", "decode", "extend", "verify"))
    hq, hkv = rng.choice(((8, 2), (32, 8), (32, 4), (64, 4), (6, 2), (8, 8)))
    kv = "fp4" if op == "fp4" else rng.choice(("bf16", "e4m3", "fp4"))
    d = 64 if kv == "bf16" and rng.random() < 0.3 else 128
    alibi, cap = False, 0.0
    if op == "bias":
        what = rng.choice(("cap", "alibi", "both"))
        alibi = what != "cap"
        cap = rng.choice((20.0, 30.0, 50.0)) if what != "alibi" else 0.0
    mix = rng.randrange(1 << 20)
    if mode == "decode":
        bs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 40, min(131071, (262144 if kv == "bf16" else 524288) // bs))
        return _attn(None, op, mode, bs, hq, hkv, d, rng.randrange(0, hi), hi, mix, 1, 1, kv, cap, alibi, page,
                     rng.randrange(0, min(bs, 3)))
    if mode == "verify":
        bs = _log_int(rng, 1, 32)
        hi = _log_int(rng, 40, min(16384, 262144 // bs))
        return _attn(None, op, mode, bs, hq, hkv, d, rng.randrange(0, hi), hi, mix, 1, rng.choice((2, 4, 8)), kv, cap,
                     alibi, page, 0, rng.choice((False, True)))
    bs = rng.randrange(1, 7)
    hi = _log_int(rng, 4, 4096)
    n_hi = _log_int(rng, 8, 800 * 32 // max(hq, 32))
    return _attn(None, op, mode, bs, hq, hkv, d, rng.randrange(0, hi), hi, mix, rng.randrange(1, n_hi), n_hi, kv, cap,
                 alibi, page)


def _lens(case):
    """Cached and new tokens of each request (the largest of each range is always there)."""
    r = random.Random(case["mix"])
    cached = [r.randint(case["lo"], case["hi"]) for _ in range(case["bs"])]
    new = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["bs"])]
    cached[-1], new[-1] = case["hi"], case["n_hi"]
    seq = [0 if b < case["empty"] else cached[b] + new[b] for b in range(case["bs"])]
    return seq, new


def _row_bytes(kv, d):
    return {"bf16": 2.0, "e4m3": 1.0, "fp4": 0.5625}[kv] * d


def work(case):
    if case["op"] == "rope":
        n, hq, hkv, dk, dv = (case[k] for k in ("tokens", "hq", "hkv", "dk", "dv"))
        pool = hkv * (_row_bytes(case["kv"], dk) + _row_bytes(case["kv"], dv))
        byte = 2 * hq * dk * 2 + hkv * (dk + dv) * 2 + pool + case["rot"] * 4 + 8
        if case["kv"] == "fp4":
            byte += hkv * (dk + dv) * 2
        return {"bytes": n * byte, "flops": n * (hq + hkv) * case["rot"] * 3}
    seq, new = _lens(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows = sum(new)
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(seq, new) if L)
    byte = sum(seq) * hkv * 2 * _row_bytes(case["kv"], d) + rows * hq * (4 * d + 4)
    byte += sum(-(-L // case["page"]) for L in seq) * 4
    return {"bytes": byte, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------- number formats
def _to_e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _fp4_codes(y):
    """E2M1 magnitude codes, signs and E4M3 block scales of scaled fp32 values [..., D]: nearest, ties to even codes."""
    blocks = y.reshape(*y.shape[:-1], y.shape[-1] // 16, 16)
    scale = _to_e4m3(blocks.abs().amax(-1) * torch.tensor(1.0 / 6.0, dtype=torch.float32, device=y.device))
    s = scale.float()
    z = blocks * torch.where(s > 0, 1.0 / s, torch.zeros_like(s)).unsqueeze(-1)
    a = z.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code.to(torch.uint8), torch.signbit(z), scale


def _fp4_values(code, negative, scale, pool_scale):
    mag = torch.tensor(E2M1_VALUES, device=code.device)[code.long()]
    v = torch.where(negative, -mag, mag) * scale.float().unsqueeze(-1)
    return v.flatten(-2) * pool_scale


def _fp4_pack(values, inv):
    """Values [slots, heads, D] as the bytes of a 4-bit pool (slots a multiple of 16)."""
    slots, h, d = values.shape
    code, negative, scale = _fp4_codes(values * inv)
    nib = (code | (negative.to(torch.uint8) << 3)).reshape(slots, h, d)
    rows = nib[..., 0::2] | (nib[..., 1::2] << 4)
    rows = rows.view(slots // 16, 16, h, d // 2).transpose(1, 2).flatten(2)
    scales = scale.view(torch.uint8).reshape(slots // 16, 16, h, d // 16).transpose(1, 2).flatten(2)
    return torch.cat([rows, scales], -1).contiguous().view(-1)


def _fp4_rows(pool, slots, h, d, pool_scale):
    """Values [*slots.shape, heads, D] of the given slots of a 4-bit pool's bytes."""
    tiles = pool.view(-1, h, 16 * (d // 2 + d // 16))
    rows = tiles[..., : 8 * d].reshape(-1, h, 16, d // 2)
    scales = tiles[..., 8 * d:].reshape(-1, h, 16, d // 16)
    seg, sub = slots // 16, slots % 16
    byte = rows.transpose(1, 2)[seg, sub]
    nib = torch.stack([byte & 15, byte >> 4], -1).flatten(-2)
    scale = scales.transpose(1, 2)[seg, sub].contiguous().view(torch.float8_e4m3fn)
    blocks = nib.reshape(*nib.shape[:-1], d // 16, 16)
    return _fp4_values(blocks & 7, blocks > 7, scale, pool_scale)


def _pool_rows(state, which, slots):
    case, pool = state["case"], state[which + "_pool"]
    if case["kv"] == "fp4":
        return _fp4_rows(pool, slots, case["hkv"], case["d"], state[which + "_scale"])
    return pool[slots].float() * state[which + "_scale"]


# ---------------------------------------------------------------- inputs
def _pages(total, page, g):
    """Page ids handed to requests in a random order; page 0 is never handed out."""
    return (torch.randperm(total, generator=g, device="cuda") + 1).to(torch.int32)


def _pool(kv, slots, heads, d, g):
    """A pool of N(0, 1) values and its scale."""
    x = torch.randn(slots, heads, d, generator=g, device="cuda")
    if kv == "bf16":
        return x.bfloat16(), 1.0
    if kv == "e4m3":
        return _to_e4m3(x / (6.0 / E4M3_MAX)), 6.0 / E4M3_MAX
    scale = 6.0 / (E4M3_MAX * E2M1_MAX)
    return _fp4_pack(x, 1.0 / scale), scale


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    state = _prepare_rope(case, g) if case["op"] == "rope" else _prepare_attention(case, g)
    if own:
        state["handle"] = _handle(state)
    return state


def _prepare_rope(case, g):
    n, hq, hkv, dk, dv, page = (case[k] for k in ("tokens", "hq", "hkv", "dk", "dv", "page"))
    qkv = torch.randn(n, hq * dk + hkv * (dk + dv), generator=g, device="cuda").bfloat16()
    pages = -(-max(n + n // 8, 256) // page) + 1
    slots = pages * page
    order = _pages(pages - 1, page, g).long()
    at = torch.arange(n, device="cuda")
    loc = (order[at // page] * page + at % page).to(torch.int32)
    # a few requests side by side, each at positions of its own
    first = torch.randint(0, 1000, (8,), generator=g, device="cuda")
    positions = (case["far"] + first[at * 8 // n] + at % 20000).to(torch.int32)
    inv_freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
    angles = torch.arange(MAX_POSITIONS, dtype=torch.float64, device="cuda")[:, None] * inv_freq
    state = dict(case=case, q=qkv[:, : hq * dk].view(n, hq, dk), k=qkv[:, hq * dk: (hq + hkv) * dk].view(n, hkv, dk),
                 v=qkv[:, (hq + hkv) * dk:].view(n, hkv, dv), loc=loc, positions=positions,
                 cos_sin=torch.cat([angles.cos(), angles.sin()], -1).float(),
                 q_out=torch.empty(n, hq, dk, dtype=torch.bfloat16, device="cuda"))
    state["k_pool"], state["k_scale"] = _pool(case["kv"], slots, hkv, dk, g)
    state["v_pool"], state["v_scale"] = _pool(case["kv"], slots, hkv, dv, g)
    state["k_rows"] = torch.empty(n, hkv, dk, dtype=torch.bfloat16, device="cuda")
    state["v_rows"] = torch.empty(n, hkv, dv, dtype=torch.bfloat16, device="cuda")
    return state


def _prepare_attention(case, g):
    bs, hq, hkv, d, page = (case[k] for k in ("bs", "hq", "hkv", "d", "page"))
    seq, new = _lens(case)
    need = [-(-L // page) for L in seq]
    total = sum(need)
    pages = total + total // 10 + 2
    order = _pages(pages - 1, page, g)
    table = torch.zeros(bs, max(max(need), 1), dtype=torch.int32)
    starts = [sum(need[:b]) for b in range(bs)]
    valid = torch.arange(table.shape[1])[None] < torch.tensor(need)[:, None]
    index = (torch.tensor(starts)[:, None] + torch.arange(table.shape[1])[None]).clamp(max=pages - 2)
    table = torch.where(valid.cuda(), order[index.cuda()], torch.zeros_like(table).cuda()).contiguous()
    rows = sum(new)
    state = dict(case=case, seq=torch.tensor(seq, dtype=torch.int32, device="cuda"),
                 new=torch.tensor(new, dtype=torch.int32, device="cuda"), table=table, pages=pages, rows=rows,
                 max_len=max(seq), max_new=max(new), pages_used=max(total, 1),
                 q=torch.randn(rows, hq, d, generator=g, device="cuda").bfloat16() * 1.5,
                 out=torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.empty(rows, hq, dtype=torch.float32, device="cuda"), sm_scale=1.0 / math.sqrt(d),
                 slopes=None)
    if case["alibi"]:
        state["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, dtype=torch.float32, device="cuda") / hq)
    state["k_pool"], state["k_scale"] = _pool(case["kv"], pages * page, hkv, d, g)
    state["v_pool"], state["v_scale"] = _pool(case["kv"], pages * page, hkv, d, g)
    return state


# ---------------------------------------------------------------- the framework's calls
def _handle(state):
    """The context that a server keeps, with the plan of the batch for attention."""
    from paged_kv_cache_15_gb300 import binding as B
    case = state["case"]
    kv = {"bf16": B.PKV_KV_BF16, "e4m3": B.PKV_KV_FP8_E4M3, "fp4": B.PKV_KV_FP4_E2M1}[case["kv"]]
    if case["op"] == "rope":
        slots = state["k_pool"].shape[0] if case["kv"] != "fp4" else state["k_pool"].numel() * 16 // (
            case["hkv"] * 9 * case["dk"])
        cfg = B.make_config(case["hq"], case["hkv"], case["dk"], case["page"], kv, slots // case["page"], 1, 1, 1, 1,
                            head_dim_v=case["dv"])
        return B.PagedAttention(cfg)
    most = max(1, min(state["max_new"], 128 // (case["hq"] // case["hkv"]))) if case["mode"] == "verify" else 1
    cfg = B.make_config(case["hq"], case["hkv"], case["d"], case["page"], kv, state["pages"], case["bs"],
                        state["pages_used"], state["rows"], most)
    attn = B.PagedAttention(cfg)
    mode = {"decode": B.PKV_MODE_DECODE, "extend": B.PKV_MODE_EXTEND, "verify": B.PKV_MODE_TARGET_VERIFY}[case["mode"]]
    state["mode"] = mode
    state["spec"] = B.PKV_SPEC_DECODE if case["tc"] else B.PKV_SPEC_PREFILL
    if case["cap"]:
        B.pkv_set_logit_cap(attn.ctx, case["cap"])
    if state["slopes"] is not None:
        B.pkv_set_alibi_slopes(attn.ctx, state["slopes"])
    B.pkv_build_metadata(attn.ctx, mode, case["bs"], state["seq"], None if case["mode"] == "decode" else state["new"],
                         state["table"])
    return attn


def _own_run(state):
    from paged_kv_cache_15_gb300 import binding as B
    case, ctx = state["case"], state["handle"].ctx
    if case["op"] == "rope":
        B.pkv_rope_set_kv_buffer(ctx, state["k_pool"], state["v_pool"], state["loc"], state["positions"],
                                 state["cos_sin"], state["q"], state["k"], state["v"], state["q_out"],
                                 rotary_offset=case["first"], interleaved=case["inter"],
                                 k_inv_scale=1.0 / state["k_scale"], v_inv_scale=1.0 / state["v_scale"])
        if case["kv"] == "fp4":
            B.pkv_get_kv_buffer(ctx, state["k_pool"], state["v_pool"], state["loc"], state["k_rows"], state["v_rows"],
                                k_scale=state["k_scale"], v_scale=state["v_scale"])
            return {"q": state["q_out"], "k_rows": state["k_rows"], "v_rows": state["v_rows"]}
        return {"q": state["q_out"], "k_pool": state["k_pool"], "v_pool": state["v_pool"]}
    B.pkv_forward(ctx, state["mode"], state["spec"], state["q"], state["k_pool"], state["v_pool"], state["sm_scale"],
                  state["out"], state["lse"], state["k_scale"], state["v_scale"])
    return {"out": state["out"], "lse": state["lse"]}


# ---------------------------------------------------------------- the plain forms
def _rotate(x, cos, sin, first, inter):
    """fp32 rows [n, heads, D] with columns first .. first + R rotated by cos, sin [n, R/2]."""
    half = cos.shape[-1]
    y = x.clone()
    part = y[..., first: first + 2 * half]
    a, b = (part[..., 0::2], part[..., 1::2]) if inter else (part[..., :half], part[..., half:])
    c, s = cos.unsqueeze(1), sin.unsqueeze(1)
    new_a, new_b = a * c - b * s, b * c + a * s
    a.copy_(new_a)
    b.copy_(new_b)
    return y


def _plain_rope(state):
    case = state["case"]
    half = case["rot"] // 2
    row = state["cos_sin"][state["positions"].long()]
    cos, sin = row[:, :half], row[:, half:]
    q = _rotate(state["q"].float(), cos, sin, case["first"], case["inter"]).bfloat16()
    k = _rotate(state["k"].float(), cos, sin, case["first"], case["inter"])
    v = state["v"].float()
    inv = {w: torch.tensor(1.0 / state[w + "_scale"], dtype=torch.float32, device="cuda") for w in ("k", "v")}
    if case["kv"] == "fp4":
        return {"q": q, **{w + "_rows": _fp4_values(*_fp4_codes(x * inv[w]), state[w + "_scale"]).bfloat16()
                           for w, x in (("k", k), ("v", v))}}
    loc = state["loc"].long()
    if case["kv"] == "e4m3":
        state["k_pool"].view(torch.uint8)[loc] = _to_e4m3(k * inv["k"]).view(torch.uint8)
        state["v_pool"].view(torch.uint8)[loc] = _to_e4m3(v * inv["v"]).view(torch.uint8)
    else:
        state["k_pool"][loc] = k.bfloat16()
        state["v_pool"][loc] = state["v"]
    return {"q": q, "k_pool": state["k_pool"], "v_pool": state["v_pool"]}


def _plain_attention(state):
    """Every request padded to the longest one: scores [bs, hkv, group, rows, keys] in fp32."""
    case = state["case"]
    bs, hq, hkv, d = case["bs"], case["hq"], case["hkv"], case["d"]
    group, page = hq // hkv, case["page"]
    seq, new = state["seq"].long(), state["new"].long()
    key = torch.arange(state["max_len"], device="cuda")
    row = torch.arange(state["max_new"], device="cuda")
    slots = state["table"].long()[:, key // page] * page + key % page
    there = key[None] < seq[:, None]
    k = _pool_rows(state, "k", slots)
    start = new.cumsum(0) - new
    at = (start[:, None] + row[None]).clamp(max=state["rows"] - 1)
    q = state["q"].float()[at].view(bs, -1, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(bs, hkv, -1, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).view(bs, hkv, group, -1, key.numel())
    del k
    s.mul_(state["sm_scale"])
    if case["cap"]:
        s.div_(case["cap"]).tanh_().mul_(case["cap"])
    last = (seq - new)[:, None] + row[None]
    if case["alibi"]:
        distance = (key[None, None] - last[..., None]).float()
        s.add_(state["slopes"].view(1, hkv, group, 1, 1) * distance[:, None, None])
    seen = (key[None, None] <= last[..., None]) & there[:, None]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    v = _pool_rows(state, "v", slots).masked_fill_(~there[:, :, None, None], 0.0)
    o = torch.matmul(s.view(bs, hkv, -1, key.numel()), v.permute(0, 2, 1, 3)).view(bs, hkv, group, -1, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(bs, -1, hq, d)
    lse = lse.permute(0, 3, 1, 2).reshape(bs, -1, hq)
    real = row[None] < new[:, None]
    return {"out": o[real].bfloat16(), "lse": lse[real]}


def run(state):
    if own:
        return _own_run(state)
    return _plain_rope(state) if state["case"]["op"] == "rope" else _plain_attention(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _round_e4m3(x):
    """fp64 values to the E4M3 grid: spacing 2^(e-3) in [2^e, 2^(e+1)), 2^-9 below 2^-6."""
    e = torch.frexp(x.abs())[1].double() - 1
    step = torch.pow(2.0, e.clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _round_fp4(x):
    """fp64 rows [..., D], block by block: scale on the E4M3 grid, values on its multiple of the E2M1 grid."""
    b = x.unflatten(-1, (-1, 16))
    s = _round_e4m3(b.abs().amax(-1, keepdim=True) / 6.0)
    z = torch.where(s > 0, b / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b))
    a = z.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return (torch.sign(z) * (torch.round(a / step) * step).clamp(max=E2M1_MAX) * s).flatten(-2)


def exact(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def rope(st):
        half, f = case["rot"] // 2, case["first"]
        table = st["cos_sin"].double()[st["positions"].long()]
        turn = torch.complex(table[:, :half], table[:, half:])[:, None]

        def turned(x):
            y = x.double().clone()
            part = y[..., f: f + case["rot"]]
            pair = part.unflatten(-1, (half, 2)) if case["inter"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            y[..., f: f + case["rot"]] = z.flatten(-2) if case["inter"] else z.transpose(-1, -2).flatten(-2)
            return y

        new = {"k": turned(st["k"]), "v": st["v"].double()}
        found = {"q": turned(st["q"])}
        for which, x in new.items():
            if case["kv"] == "fp4":
                found[which + "_rows"] = _round_fp4(x / st[which + "_scale"]) * st[which + "_scale"]
            else:
                pool = st[which + "_pool"].double()
                pool[st["loc"].long()] = _round_e4m3(x / st[which + "_scale"]) if case["kv"] == "e4m3" else x
                found[which + "_pool"] = pool
        return found

    def attention(st):
        seq, new = _lens(case)
        hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
        out = torch.zeros(sum(new), hq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((sum(new), hq), -math.inf, dtype=torch.float64, device="cuda")
        t0 = 0
        for b, (L, n) in enumerate(zip(seq, new)):
            if L:
                pos = torch.arange(L, device="cuda")
                slots = st["table"][b].long()[pos // page] * page + pos % page
                k, v = (_pool_rows(st, w, slots).double() for w in ("k", "v"))
                row = torch.arange(L - n, L, device="cuda")[:, None]
                for h in range(hq):
                    s = st["q"][t0: t0 + n, h].double() @ k[:, h * hkv // hq].T * st["sm_scale"]
                    if case["cap"]:
                        s = case["cap"] * torch.tanh(s / case["cap"])
                    if case["alibi"]:
                        s = s + st["slopes"][h].double() * (pos[None] - row).double()
                    s = s.masked_fill(pos[None] > row, -math.inf)
                    lse[t0: t0 + n, h] = torch.logsumexp(s, -1)
                    out[t0: t0 + n, h] = torch.softmax(s, -1) @ v[:, h * hkv // hq]
            t0 += n
        return {"out": out, "lse": lse}

    return rope(_prepare_rope(case, g)) if case["op"] == "rope" else attention(_prepare_attention(case, g))
