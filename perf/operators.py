"""The operators of a paged serving and training step around attention, as measurable cases.

Five operators, each in a plain form (elementary torch operations in 32 bits, `own` false) and
through the package's entry points (`own` true):

  slots       block tables, slot maps, offsets and positions of a step from its request lengths
  rope        RMS norm of queries and keys per head, with the position rotation (one or more axes)
  rope_bwd    its gradients (queries, keys and both norm weights)
  store       new keys and values into pages of the 4-bit cache, and the same rows read back
  attend      attention of packed queries over that cache

The 4-bit cache holds e2m1 codes (two a byte, the even element in the low nibble) with one e4m3
scale for 16 elements and one fp32 descale a tensor: value = code * scale * descale.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MAX_PAST = 131072


def _lengths(n, lo, hi, seed):
    """n whole lengths, log-uniform in [lo, hi]."""
    r = random.Random(seed)
    lo1, hi1 = max(1, lo), max(1, hi)
    got = [round(math.exp(math.log(lo1) + r.random() * (math.log(hi1) - math.log(lo1)))) for _ in range(n)]
    return [lo if lo == hi else max(lo, min(hi, x)) for x in got]


def listed():
    return [
        # one decoding step of 128 requests with caches of 1K to 32K tokens
        {"name": "slots_decode_128", "op": "slots", "n": 128, "past_lo": 1024, "past_hi": 32768, "new_lo": 1, "new_hi": 1,
         "page": 64, "lens_seed": 12},
        # a prefill step of 32 prompts of 512 to 8192 tokens, small pages
        {"name": "slots_prefill_32", "op": "slots", "n": 32, "past_lo": 0, "past_hi": 0, "new_lo": 512, "new_hi": 8192,
         "page": 16, "lens_seed": 11},
        # one decoding step: 128 tokens, 32 query heads on 8 key/value heads
        {"name": "rope_decode_128", "op": "rope", "batch": 1, "seq": 128, "H": 32, "H_kv": 8, "D": 128, "rot": 128, "axes": 1,
         "interleaved": False, "norm": True, "dtype": "bf16", "fused": True},
        # images and text: three position axes, 4 x 4096 tokens out of a fused projection
        {"name": "rope_3axes_4x4096", "op": "rope", "batch": 4, "seq": 4096, "H": 32, "H_kv": 8, "D": 128, "rot": 128, "axes": 3,
         "interleaved": False, "norm": True, "dtype": "bf16", "fused": True},
        # an odd length, half of each head rotated in neighbouring pairs, fp16
        {"name": "rope_partial_2x4097", "op": "rope", "batch": 2, "seq": 4097, "H": 16, "H_kv": 16, "D": 64, "rot": 32, "axes": 1,
         "interleaved": True, "norm": True, "dtype": "f16", "fused": False},
        # training: the gradients at 4 x 4096 tokens
        {"name": "rope_bwd_4x4096", "op": "rope_bwd", "batch": 4, "seq": 4096, "H": 32, "H_kv": 8, "D": 128, "rot": 128, "axes": 1,
         "interleaved": False, "norm": True, "dtype": "bf16", "fused": True},
        # a short fine-tuning batch, odd length, fp16
        {"name": "rope_bwd_2x257", "op": "rope_bwd", "batch": 2, "seq": 257, "H": 8, "H_kv": 2, "D": 64, "rot": 64, "axes": 3,
         "interleaved": True, "norm": True, "dtype": "f16", "fused": False},
        # one new token of each of 128 requests
        {"name": "store_decode_128", "op": "store", "tokens": 128, "H_kv": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # the new tokens of a chunked prefill, 8 x 1024
        {"name": "store_prefill_8192", "op": "store", "tokens": 8192, "H_kv": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # decoding, 4 short requests, small pages, fp16, heads of 64
        {"name": "attend_decode_4", "op": "attend", "n": 4, "k_lo": 300, "k_hi": 2000, "q_lo": 1, "q_hi": 1, "H": 16, "H_kv": 4,
         "D": 64, "page": 16, "dtype": "f16", "lens_seed": 3},
        # decoding, 128 requests with caches of 1K to 32K tokens
        {"name": "attend_decode_128", "op": "attend", "n": 128, "k_lo": 1024, "k_hi": 32768, "q_lo": 1, "q_hi": 1, "H": 32,
         "H_kv": 8, "D": 128, "page": 64, "dtype": "bf16", "lens_seed": 12},
        # chunked prefill: 1024 new tokens after 7168 held ones, 8 requests
        {"name": "attend_prefill_8x1024", "op": "attend", "n": 8, "k_lo": 8192, "k_hi": 8192, "q_lo": 1024, "q_hi": 1024, "H": 32,
         "H_kv": 8, "D": 128, "page": 64, "dtype": "bf16", "lens_seed": 1},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["slots", "rope", "rope_bwd", "store", "attend", "attend"])
    heads = rng.choice([(32, 8), (16, 16), (8, 2), (16, 4), (8, 1), (12, 4), (28, 4), (64, 8)])
    dim = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    if op == "slots":
        if rng.random() < 0.5:
            return {"op": op, "n": log_int(1, 1024), "past_lo": 0, "past_hi": log_int(16, 32768), "new_lo": 1, "new_hi": rng.choice([1, 1, 4]),
                    "page": rng.choice([16, 32, 64, 128]), "lens_seed": rng.randrange(1 << 20)}
        hi = log_int(16, 8192)
        return {"op": op, "n": log_int(1, 32), "past_lo": 0, "past_hi": rng.choice([0, 1000, 20000]), "new_lo": max(1, hi // 16), "new_hi": hi,
                "page": rng.choice([16, 32, 64, 128]), "lens_seed": rng.randrange(1 << 20)}
    if op in ("rope", "rope_bwd"):
        most = 16384 * 40 * 128 // ((heads[0] + heads[1]) * dim)
        tokens = log_int(1, most)
        batch = rng.choice([1, 2, 4])
        rot = rng.choice([dim, dim, dim // 2, 16])
        return {"op": op, "batch": batch, "seq": max(1, tokens // batch), "H": heads[0], "H_kv": heads[1], "D": dim, "rot": rot,
                "axes": rng.choice([1, 1, 2, 3]), "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.8, "dtype": dtype,
                "fused": rng.random() < 0.5}
    if op == "store":
        return {"op": op, "tokens": log_int(1, 8192), "H_kv": heads[1] if heads[1] <= 8 else 8, "D": dim, "page": rng.choice([16, 32, 64, 128]), "dtype": dtype}
    n = log_int(1, 64)
    k_hi = log_int(16, 32768)
    kind = rng.choice(["decode", "decode", "few", "chunk"])
    q_hi = {"decode": 1, "few": rng.choice([2, 4, 8]), "chunk": log_int(9, 1024)}[kind]
    if kind == "chunk":
        n, k_hi = max(1, min(n, 8)), max(min(k_hi, 8192), q_hi)
        heads = heads if heads[0] <= 32 else (32, 8)
    n = max(1, min(n, (1 << 30) // (k_hi * heads[1] * dim)))
    return {"op": op, "n": n, "k_lo": max(1, k_hi // rng.choice([1, 4, 16])), "k_hi": k_hi, "q_lo": max(1, q_hi // rng.choice([1, 4])), "q_hi": q_hi,
            "H": heads[0], "H_kv": heads[1], "D": dim, "page": rng.choice([16, 32, 64, 128]), "dtype": dtype, "lens_seed": rng.randrange(1 << 20)}


# ---------------------------------------------------------------- sizes

def _slots_sizes(c):
    past = _lengths(c["n"], c["past_lo"], c["past_hi"], c["lens_seed"])
    new = _lengths(c["n"], c["new_lo"], c["new_hi"], c["lens_seed"] + 1)
    ps = c["page"]
    have = [-(-p // ps) for p in past]
    need = [-(-(p + m) // ps) for p, m in zip(past, new)]
    rows = -(-sum(new) // 64) * 64                     # a batch padded to whole 64 rows
    return past, new, have, need, max(need), rows


def _attend_sizes(c):
    k = _lengths(c["n"], c["k_lo"], c["k_hi"], c["lens_seed"])
    q = [min(a, b) for a, b in zip(_lengths(c["n"], c["q_lo"], c["q_hi"], c["lens_seed"] + 1), k)]
    return q, k


def _axis_of_pair(c):
    """The axis of each rotated pair: a quarter for the first, the rest in equal runs."""
    pairs, axes = c["rot"] // 2, c["axes"]
    first = pairs if axes == 1 else max(1, pairs // 4)
    rest = pairs - first
    return [0 if i < first else 1 + (i - first) * (axes - 1) // max(1, rest) for i in range(pairs)]


def work(case):
    c = case
    if c["op"] == "slots":
        past, new, have, need, cols, rows = _slots_sizes(c)
        taken = sum(b - a for a, b in zip(have, need))
        # lengths and free pages in; offsets, new table entries, positions and slots out
        return {"bytes": 4.0 * (4 * c["n"] + 2 * taken) + 12.0 * rows, "flops": 8.0 * rows}
    if c["op"] in ("rope", "rope_bwd"):
        t, heads = c["batch"] * c["seq"], c["H"] + c["H_kv"]
        b = 2.0 * t * heads * c["D"]
        passes = 2 if c["op"] == "rope" or not c["norm"] else 3
        return {"bytes": passes * b + 4.0 * t * c["axes"] + 8.0 * c["D"], "flops": (8.0 if c["op"] == "rope" else 16.0) * t * heads * c["D"]}
    if c["op"] == "store":
        e = 2.0 * c["tokens"] * c["H_kv"] * c["D"]
        # 16-bit rows in, codes and scales out, then codes and scales in and 16-bit rows out
        return {"bytes": 2 * (2 * e + e * 9 / 16) + 16.0 * c["tokens"], "flops": 6.0 * e}
    q, k = _attend_sizes(c)
    held = 2.0 * sum(k) * c["H_kv"] * c["D"] * 9 / 16
    seen = sum(sum(min(b, b - a + i + 1) for i in range(a)) for a, b in zip(q, k))
    return {"bytes": held + 4.0 * sum(q) * c["H"] * c["D"] + 4.0 * sum(q) * c["H"], "flops": 4.0 * seen * c["H"] * c["D"]}


# ---------------------------------------------------------------- inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _to_cache(x, descale):
    """Codes and e4m3 scales of x [..., D], by the format's rule: each group's scale is the e4m3 value nearest to
    amax / (6 descale), each code the e2m1 value nearest to x / (scale descale), ties to the even one. In 64 bits:
    the inputs are 16-bit values, so that many lie next to a border or on it."""
    shape = x.shape
    x = x.reshape(-1, shape[-1] // 16, 16).double()
    g = descale.double()
    want = x.abs().amax(-1) / (6.0 * g)
    step = torch.exp2((torch.frexp(want)[1] - 1).clamp_(min=-6).double() - 3.0)
    scale = (torch.round(want / step) * step).clamp_(max=448.0)
    y = torch.where((scale > 0).unsqueeze(-1), x / (scale * g).unsqueeze(-1), torch.zeros_like(x))
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    code = code + torch.signbit(y).to(torch.uint8) * 8
    code = code.reshape(-1, shape[-1] // 2, 2)
    codes = (code[..., 0] | (code[..., 1] << 4)).reshape(*shape[:-1], shape[-1] // 2)
    return codes, scale.to(torch.float8_e4m3fn).reshape(*shape[:-1], shape[-1] // 16)


def _values(codes, scales, descale):
    """The fp32 values that codes [..., D / 2] and scales [..., D / 16] stand for."""
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], codes.shape[-1] * 2).long()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    v = table[c].reshape(*scales.shape, 16) * (scales.float() * descale).unsqueeze(-1)
    return v.reshape(c.shape)


def _make_cache(pages, c, g, fill):
    shape = (pages, c["H_kv"], c["page"], c["D"])
    st = {}
    for name, std in (("k", 1.0), ("v", 0.7)):
        codes = torch.zeros(*shape[:-1], c["D"] // 2, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(*shape[:-1], c["D"] // 16, dtype=torch.float8_e4m3fn, device="cuda")
        # the descale that puts the largest values in the e4m3 scale's upper range
        descale = torch.tensor([6.5 * std / (6.0 * 448.0)], dtype=torch.float32, device="cuda")
        if fill:
            per = max(1, (1 << 25) // math.prod(shape[1:]))
            for a in range(0, pages, per):
                x = torch.randn((min(per, pages - a),) + shape[1:], generator=g, device="cuda") * std
                codes[a:a + per], got = _to_cache(x, descale)
                scales[a:a + per] = got
        st[name + "_codes"], st[name + "_scales"], st[name + "_descale"] = codes, scales, descale
    return st


def prepare(case, seed):
    c = case
    g = _gen(seed)
    s = {"case": c}
    if c["op"] == "slots":
        past, new, have, need, cols, rows = _slots_sizes(c)
        pages = sum(need) + 17
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((c["n"], cols), -7, dtype=torch.int32, device="cuda")
        held = torch.arange(cols, device="cuda")[None, :] < torch.tensor(have, device="cuda")[:, None]
        table[held] = order[: sum(have)]
        s.update(past=torch.tensor(past, dtype=torch.int32, device="cuda"), new=torch.tensor(new, dtype=torch.int32, device="cuda"),
                 free=order[sum(have):].contiguous(), table=table, rows=rows,
                 out=dict(cu_seqlens_q=torch.empty(c["n"] + 1, dtype=torch.int32, device="cuda"),
                          seqused_k=torch.empty(c["n"], dtype=torch.int32, device="cuda"),
                          positions=torch.empty(rows, dtype=torch.int32, device="cuda"),
                          slot_map=torch.empty(rows, dtype=torch.int64, device="cuda"),
                          pages_taken=torch.empty(1, dtype=torch.int32, device="cuda")))
        if own:
            from tiled_attention_10_gb300 import PagedSlots
            s["out"] = PagedSlots(**s["out"])
        return s
    if c["op"] in ("rope", "rope_bwd"):
        b, t, h, hk, d = c["batch"], c["seq"], c["H"], c["H_kv"], c["D"]
        dt = DTYPES[c["dtype"]]

        def rows(heads):
            return torch.randn(b, t, heads, d, generator=g, device="cuda").to(dt)

        def pair():
            if c["fused"]:                              # views of one projection's output [B, S, H + 2 H_kv, D]
                x = rows(h + 2 * hk)
                return x[:, :, :h], x[:, :, h:h + hk]
            return rows(h), rows(hk)

        s["q"], s["k"] = pair()
        s["wq"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if c["norm"] else None
        s["wk"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if c["norm"] else None
        start = torch.randint(0, MAX_PAST, (c["axes"], b, 1), generator=g, device="cuda")
        line = torch.arange(t, device="cuda")
        pos = [start[0] + line]                         # time; then rows and columns of a 32-wide image
        pos += [start[i] % 1024 + (line // 32 if i == 1 else line % 32) for i in range(1, c["axes"])]
        s["pos"] = torch.stack(pos).to(torch.int32).contiguous()
        s["inv_freq"] = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        s["axis_list"] = _axis_of_pair(c)
        s["axis"] = torch.tensor(s["axis_list"], device="cuda")
        s["pair_axis"] = s["axis_list"] if c["axes"] > 1 else None
        if c["op"] == "rope_bwd":
            s["dq"], s["dk"] = rows(h), rows(hk)
        return s
    if c["op"] == "store":
        n, hk, d, ps = c["tokens"], c["H_kv"], c["D"], c["page"]
        pages = -(-n // ps) + 5
        s.update(_make_cache(pages, c, g, False))
        x = torch.randn(n, hk + 2 * hk, d, generator=g, device="cuda").to(DTYPES[c["dtype"]])
        s["k"], s["v"] = x[:, hk:2 * hk], x[:, 2 * hk:]
        # runs of consecutive slots in shuffled pages; every 61st row is padding
        page = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        s["slots"] = torch.where(t % 61 == 60, torch.full_like(t, -1), page[t // ps] * ps + t % ps)
        s["k_out"], s["v_out"] = (torch.empty(n, hk, d, dtype=DTYPES[c["dtype"]], device="cuda") for _ in range(2))
    else:
        q, k = _attend_sizes(c)
        ps = c["page"]
        per = [-(-x // ps) for x in k]
        order = torch.randperm(sum(per), generator=g, device="cuda").to(torch.int32)
        s.update(_make_cache(sum(per), c, g, True))
        table = torch.full((c["n"], max(per)), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(max(per), device="cuda")[None, :] < torch.tensor(per, device="cuda")[:, None]] = order
        s["table"], s["q_len"], s["k_len"] = table, q, k
        s["seqused_k"] = torch.tensor(k, dtype=torch.int32, device="cuda")
        cu = [0]
        for x in q:
            cu.append(cu[-1] + x)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["q"] = torch.randn(cu[-1], c["H"], c["D"], generator=g, device="cuda").to(DTYPES[c["dtype"]])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(c["H"], cu[-1], dtype=torch.float32, device="cuda")
        s["max_q"], s["max_k"], s["total_k"] = max(q), max(k), sum(k)
        s["scale"] = c["D"] ** -0.5
    if own:
        from tiled_attention_10_gb300 import KV4Cache, paged_attention_kv4_workspace
        s["cache"] = KV4Cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["k_descale"], s["v_descale"])
        if c["op"] == "attend":
            s["workspace"] = paged_attention_kv4_workspace(s["q"], s["cache"], max_seqlen_q=s["max_q"], n_seqs=c["n"], total_k=s["total_k"])
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import tiled_attention_10_gb300 as fa
        if op == "slots":
            o = fa.paged_slots(s["past"], s["new"], s["free"], s["table"], page_size=s["case"]["page"], total_q=s["rows"], out=s["out"])
            return [o.cu_seqlens_q, o.seqused_k, o.positions, o.slot_map, o.pages_taken, s["table"]]
        if op == "rope":
            return fa.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"], norm=s["case"]["norm"], eps=1e-6,
                                   pair_axis=s["pair_axis"], interleaved=s["case"]["interleaved"], layout="BSND")
        if op == "rope_bwd":
            return fa.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"],
                                            norm=s["case"]["norm"], eps=1e-6, pair_axis=s["pair_axis"], interleaved=s["case"]["interleaved"],
                                            layout="BSND")
        if op == "store":
            fa.kv4_write(s["k"], s["v"], s["slots"], s["cache"])
            return fa.kv4_read(s["cache"], s["slots"], out=(s["k_out"], s["v_out"]))
        return fa.paged_attention_kv4(s["q"], s["cache"], s["cu"], s["seqused_k"], s["table"], max_seqlen_q=s["max_q"], total_k=s["total_k"],
                                      scale=s["scale"], causal="bottom_right", out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"slots": _slots_plain, "rope": _rope_plain, "rope_bwd": _rope_bwd_plain, "store": _store_plain, "attend": _attend_plain}[op](s)


def _slots_plain(s):
    ps, rows, table = s["case"]["page"], s["rows"], s["table"]
    past, new = s["past"].long().clamp(min=0), s["new"].long().clamp(min=0)
    n, cols = table.shape
    past = past.clamp(max=cols * ps)
    used = (past + new).clamp(max=cols * ps)
    have, end = (past + ps - 1) // ps, (used + ps - 1) // ps
    before = torch.cumsum(end - have, 0) - (end - have)
    col = torch.arange(cols, device=table.device)[None, :]
    at = before[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < end[:, None])
    page = torch.where(at < s["free"].numel(), s["free"][at.clamp(0, s["free"].numel() - 1)], torch.full_like(table, -1))
    table.copy_(torch.where(fresh, page, table))
    cu = torch.zeros(n + 1, dtype=torch.int64, device=table.device)
    cu[1:] = torch.cumsum(new, 0)
    t = torch.arange(rows, device=table.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = seq < n
    seq = seq.clamp(max=n - 1)
    pos = past[seq] + t - cu[seq]
    held = table[seq, (pos // ps).clamp(max=cols - 1)].long()
    slot = torch.where(real & (pos < cols * ps) & (held >= 0), held * ps + pos % ps, torch.full_like(pos, -1))
    return [cu.clamp(max=rows).int(), used.int(), torch.where(real, pos, torch.zeros_like(pos)).int(), slot, (end - have).sum().int().reshape(1), table]


def _angles(s):
    """cos and sin of each token's pairs, [B, S, 1, rot / 2], the angles in 64 bits."""
    a = s["pos"].double()[s["axis"]].permute(1, 2, 0) * s["inv_freq"]
    return a.cos().float().unsqueeze(2), a.sin().float().unsqueeze(2)


def _turn(x, cos, sin, rot, interleaved):
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _rope_plain(s):
    c = s["case"]
    cos, sin = _angles(s)
    got = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.float()
        if c["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        got.append(_turn(y, cos, sin, c["rot"], c["interleaved"]).to(x.dtype))
    return got


def _rope_bwd_plain(s):
    c = s["case"]
    cos, sin = _angles(s)
    grads, weights = [], []
    for dy, x, w in ((s["dq"], s["q"], s["wq"]), (s["dk"], s["k"], s["wk"])):
        g = _turn(dy.float(), cos, -sin, c["rot"], c["interleaved"])
        if not c["norm"]:
            grads.append(g.to(x.dtype))
            weights.append(None)
            continue
        y = x.float()
        r = torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
        y = y * r
        u = g * w.float()
        grads.append((r * (u - y * (u * y).mean(-1, keepdim=True))).to(x.dtype))
        weights.append((g * y).flatten(0, 2).sum(0).to(w.dtype))
    return grads + weights


def _store_plain(s):
    ps, slots = s["case"]["page"], s["slots"]
    real = (slots >= 0) & (slots < s["k_codes"].shape[0] * ps)
    page, row = slots.clamp(min=0) // ps, slots.clamp(min=0) % ps
    got = []
    for x, name in ((s["k"], "k"), (s["v"], "v")):
        codes, scales = _to_cache(x, s[name + "_descale"])
        s[name + "_codes"][page[real], :, row[real]] = codes[real]
        s[name + "_scales"].view(torch.uint8)[page[real], :, row[real]] = scales.view(torch.uint8)[real]
        y = _values(s[name + "_codes"][page, :, row], s[name + "_scales"].view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn), s[name + "_descale"])
        got.append(torch.where(real[:, None, None], y, torch.zeros_like(y)).to(x.dtype))
    return got


def _attend_plain(s):
    c = s["case"]
    h, hk, d, ps = c["H"], c["H_kv"], c["D"], c["page"]
    at = 0
    for i, (ql, kl) in enumerate(zip(s["q_len"], s["k_len"])):
        pages = s["table"][i, : -(-kl // ps)].long()
        k, v = (_values(s[n + "_codes"][pages], s[n + "_scales"].view(torch.uint8)[pages].view(torch.float8_e4m3fn), s[n + "_descale"])
                .transpose(0, 1).reshape(hk, -1, d)[:, :kl] for n in ("k", "v"))
        q = s["q"][at:at + ql].float().reshape(ql, hk, h // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
        a = (q @ k.transpose(1, 2) * s["scale"]).reshape(h, ql, kl)
        if ql > 1:
            hidden = torch.arange(kl, device=a.device)[None, :] > torch.arange(ql, device=a.device)[:, None] + (kl - ql)
            a = a.masked_fill(hidden, -math.inf)
        top = a.amax(-1, keepdim=True)
        a = (a - top).exp()
        total = a.sum(-1, keepdim=True)
        o = (a / total).reshape(hk, -1, kl) @ v
        s["out"][at:at + ql] = o.reshape(h, ql, d).transpose(0, 1).to(s["q"].dtype)
        s["lse"][:, at:at + ql] = (top + total.log()).squeeze(-1)
        at += ql
    return s["out"], s["lse"]


# ---------------------------------------------------------------- 64 bits

def _decode64(codes, scales):
    """codes * scales in 64 bits, from the bits: sign, two exponent bits (bias 1), one mantissa bit."""
    c = torch.empty(*codes.shape[:-1], codes.shape[-1], 2, dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        n = (codes.int() >> (4 * half)) & 15
        e, m = (n >> 1) & 3, (n & 1).double()
        v = torch.where(e == 0, m * 0.5, (1.0 + m * 0.5) * 2.0 ** (e.double() - 1.0))
        c[..., half] = torch.where(n >= 8, -v, v)
    c = c.flatten(-2)
    b = scales.view(torch.uint8).int()
    e, m = (b >> 3) & 15, (b & 7).double()
    f = torch.where(e == 0, m / 8.0 * 2.0 ** -6, (1.0 + m / 8.0) * 2.0 ** (e.double() - 7.0))
    return c * f.repeat_interleave(16, -1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = s["case"]
    if c["op"] == "slots":
        return None                                     # whole numbers
    if c["op"] in ("rope", "rope_bwd"):
        ang = torch.empty(*s["pos"].shape[1:], c["rot"] // 2, dtype=torch.float64, device="cuda")
        for i, ax in enumerate(s["axis_list"]):
            ang[..., i] = s["pos"][ax].double() * float(s["inv_freq"][i])
        z = torch.polar(torch.ones_like(ang), ang).unsqueeze(2)

        def forward(x, w):
            if c["norm"]:
                x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w
            r, rest = x[..., : c["rot"]], x[..., c["rot"]:]
            if c["interleaved"]:
                y = torch.view_as_complex(r.reshape(*r.shape[:-1], -1, 2).contiguous()) * z
                y = torch.view_as_real(y).flatten(-2)
            else:
                half = c["rot"] // 2
                y = torch.complex(r[..., :half], r[..., half:]) * z
                y = torch.cat((y.real, y.imag), -1)
            return torch.cat((y, rest), -1)

        if c["op"] == "rope":
            return [forward(s["q"].double(), s["wq"].double() if c["norm"] else None), forward(s["k"].double(), s["wk"].double() if c["norm"] else None)]
        gx, gw = [], []
        for dy, x, w in ((s["dq"], s["q"], s["wq"]), (s["dk"], s["k"], s["wk"])):
            x = x.double().requires_grad_()
            leaves = [x] + ([w.double().requires_grad_()] if c["norm"] else [])
            g = torch.autograd.grad(forward(x, leaves[-1]), leaves, dy.double())
            gx.append(g[0])
            gw.append(g[1] if c["norm"] else None)
            del x, leaves, g
        return gx + gw
    if c["op"] == "store":
        got = []
        grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        for x, name in ((s["k"], "k"), (s["v"], "v")):
            x = x.double()
            g = s[name + "_descale"].double()
            y = x.reshape(*x.shape[:-1], -1, 16)
            want = y.abs().amax(-1) / (6.0 * g)
            # the nearest e4m3 value: 3 mantissa bits above 2^-6, steps of 2^-9 below
            step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3.0)
            f = ((want / step).round() * step).clamp(max=448.0)
            t = (f * g).unsqueeze(-1)
            z = torch.where(t > 0, y.abs() / t, torch.zeros_like(y))
            low = (torch.searchsorted(grid, z, right=True) - 1).clamp(0, 6)
            lo, hi = grid[low], grid[low + 1]
            up = (z - lo > hi - z) | ((z - lo == hi - z) & (low % 2 == 1))
            v = torch.where(up, hi, lo) * t * torch.sign(y)
            v = v.reshape(x.shape)
            got.append(torch.where(((s["slots"] >= 0))[:, None, None], v, torch.zeros_like(v)))
        return got
    h, hk, d, ps = c["H"], c["H_kv"], c["D"], c["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (ql, kl) in enumerate(zip(s["q_len"], s["k_len"])):
        pages = s["table"][i, : -(-kl // ps)].long()
        rows = torch.arange(at, at + ql, device="cuda")
        last = kl - ql + torch.arange(ql, device="cuda")
        for j in range(hk):
            k = _decode64(s["k_codes"][pages, j], s["k_scales"].view(torch.uint8)[pages, j]).reshape(-1, d)[:kl] * s["k_descale"].double()
            v = _decode64(s["v_codes"][pages, j], s["v_scales"].view(torch.uint8)[pages, j]).reshape(-1, d)[:kl] * s["v_descale"].double()
            for m in range(j * (h // hk), (j + 1) * (h // hk)):
                a = s["q"][rows, m].double() @ k.t() * s["scale"]
                a = torch.where(torch.arange(kl, device="cuda")[None, :] <= last[:, None], a, torch.full_like(a, -math.inf))
                l = torch.logsumexp(a, -1)
                out[rows, m] = torch.exp(a - l[:, None]) @ v
                lse[m, rows] = l
        at += ql
    return [out, lse]
