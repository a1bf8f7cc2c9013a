"""Measured cases of the operators over a KV cache held in 4 bits: the append
that quantises (plain and rotating), the read-back of cached rows, and the
attention that reads the pools.

A page of 4-bit K (or V) is one run of bytes: the codes [P, Hk, D/2] (HND:
[Hk, P, D/2]), element 2i in the low half of byte i, then one 32-bit word for
each group of elements of a head, [P, Hk, G] (HND: [Hk, P, G]), a bf16 step in
its low half and a bf16 origin in its high half, padded to 16 bytes.  A code c
stands for origin + step * c.

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, through the library's entry points.  ``exact`` gives the outputs in 64
bits, written apart from both.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the rows of one decode step of 64 requests, quantised into the cache and read
        # back as attention sees them
        dict(name="append decode 64", op="append", batch=64, new_lo=1, new_hi=1, prefix_hi=4096,
             mix=1, page=16, layout="NHD", kv="int4_g128", q_heads=32, k_heads=8, dim=128),
        # the benchmark's append-prefill step (16 requests of 128..1024 new rows) in
        # the smallest groups
        dict(name="append prefill", op="append", batch=16, new_lo=128, new_hi=1024,
             prefix_hi=4096, mix=2, page=16, layout="HND", kv="int4_g32", q_heads=32, k_heads=8,
             dim=128),
        # a decode step of 256 requests that rotates on its way into the cache
        dict(name="rope_append decode 256", op="rope_append", batch=256, new_lo=1, new_hi=1,
             prefix_hi=1000, mix=3, pad=0, page=16, layout="HND", kv="int4_g64", q_heads=32,
             k_heads=8, dim=128, rotary=128, interleaved=False, scaling="parts", fused=True),
        # a prompt's rows as a captured step sees them: the buffers end in rows of no
        # request
        dict(name="rope_append prefill", op="rope_append", batch=16, new_lo=128, new_hi=1024,
             prefix_hi=4096, mix=2, pad=61, page=16, layout="NHD", kv="int4_g128", q_heads=32,
             k_heads=8, dim=128, rotary=128, interleaved=False, scaling="parts", fused=True),
        # the few rows of a short request, for a copy in full precision
        dict(name="read 17 rows", op="read", batch=1, len_lo=17, len_hi=17, mix=4, page=1,
             layout="NHD", kv="int4_g32", q_heads=4, k_heads=2, dim=64),
        # the histories of 16 requests, as work on whole prompts takes them
        dict(name="read 16 histories", op="read", batch=16, len_lo=512, len_hi=5120, mix=5,
             page=16, layout="NHD", kv="int4_g64", q_heads=32, k_heads=8, dim=128),
        # the same of 8-bit pools
        dict(name="read e4m3 histories", op="read", batch=16, len_lo=512, len_hi=5120, mix=5,
             page=16, layout="HND", kv="e4m3", q_heads=32, k_heads=8, dim=128),
        # the first token after a short prompt: latency alone
        dict(name="decode 1 of 17", op="attend", batch=1, new_lo=1, new_hi=1, kv_lo=17, kv_hi=17,
             mix=6, page=16, layout="NHD", kv="int4_g128", q_heads=32, k_heads=8, dim=128),
        # the benchmark's batch decode: 64 requests of 512..4096 keys
        dict(name="decode 64", op="attend", batch=64, new_lo=1, new_hi=1, kv_lo=512, kv_hi=4096,
             mix=7, page=16, layout="NHD", kv="int4_g128", q_heads=32, k_heads=8, dim=128),
        # the long histories of the mixed serving step: 8 requests of 32K..128K keys
        dict(name="decode 8 of 128K", op="attend", batch=8, new_lo=1, new_hi=1, kv_lo=32768,
             kv_hi=131072, mix=8, page=16, layout="HND", kv="int4_g64", q_heads=32, k_heads=8,
             dim=128),
        # a token pool (page size 1), small heads, seven of them
        dict(name="decode token pool", op="attend", batch=37, new_lo=1, new_hi=1, kv_lo=1,
             kv_hi=6001, mix=9, page=1, layout="NHD", kv="int4_g32", q_heads=28, k_heads=7,
             dim=64),
        # the benchmark's append-prefill attention: 128..1024 causal rows a request
        dict(name="prefill 16", op="attend", batch=16, new_lo=128, new_hi=1024, kv_lo=128,
             kv_hi=5120, mix=10, page=16, layout="HND", kv="int4_g128", q_heads=32, k_heads=8,
             dim=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rope_append", "read", "attend", "attend", "attend"])
    dim = rng.choice([64, 128])
    q_heads, k_heads = rng.choice([(8, 1), (8, 2), (32, 8), (8, 8), (28, 7), (5, 5), (32, 4)])
    kv = rng.choice(["int4_g32", "int4_g64"] + ["int4_g128"] * (dim == 128))
    case = dict(op=op, mix=rng.randint(0, 1 << 30), page=rng.choice([1, 3, 4, 8, 16, 64]),
                layout=rng.choice(["NHD", "HND"]), kv=kv, q_heads=q_heads, k_heads=k_heads,
                dim=dim)
    if op in ("append", "rope_append"):
        batch = _log(rng, 1, 256)
        new_hi = 1 if rng.random() < 0.5 else max(1, _log(rng, 1, 9000) // batch)
        case.update(batch=batch, new_lo=min(new_hi, rng.randint(batch <= 4, 2)), new_hi=new_hi,
                    prefix_hi=min(_log(rng, 16, 4096), 100000 // batch))
        if op == "rope_append":
            case.update(pad=rng.choice([0, 0, rng.randint(1, 64)]),
                        rotary=rng.choice([dim, dim, dim // 2, dim // 4,
                                           2 * rng.randint(1, dim // 2)]),
                        interleaved=rng.random() < 0.5,
                        scaling=rng.choice(["none", "linear", "parts"]),
                        fused=rng.random() < 0.5)
        return case
    if op == "read":
        batch = _log(rng, 1, 64)
        len_hi = max(1, min(_log(rng, 1, 8192), 80000 // batch))
        case.update(batch=batch, len_lo=rng.randint(1, len_hi), len_hi=len_hi,
                    kv=rng.choice([kv, kv, "e4m3", "bf16"]))
        return case
    # decode steps, the verification of a few drafted tokens, and chunks of prompts
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    if kind == "decode":
        batch = _log(rng, 1, 256)
        kv_hi = max(2, min(_log(rng, 1, 131072), 600000 // batch))
        new = (1, 1)
    elif kind == "verify":
        batch = _log(rng, 1, 64)
        kv_hi = max(16, min(_log(rng, 16, 16384), 100000 // batch))
        new = (rng.randint(1, 3), rng.randint(3, 8))
    else:
        batch = _log(rng, 1, 16)
        new_hi = max(2, min(_log(rng, 2, 1024), 8192 // batch))
        new = (rng.randint(1, new_hi), new_hi)
        kv_hi = max(new_hi, min(_log(rng, 16, 5120), 40000 // batch))
    case.update(batch=batch, new_lo=new[0], new_hi=new[1], kv_lo=rng.randint(1, kv_hi),
                kv_hi=kv_hi)
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

ROPE_SCALING = {
    "none": dict(base=10000.0),
    "linear": dict(base=10000.0, scaling="linear", factor=4.0),
    "parts": dict(base=500000.0, scaling="parts", factor=8.0, original_len=8192.0,
                  low_rotations=1.0, high_rotations=32.0,
                  magnitude=0.1 * math.log(8.0) + 1.0),
}

#: The scales of 8-bit K and V.
SCALES = {"e4m3": (0.03125, 0.02)}


def _group(case):
    return int(case["kv"][6:]) if case["kv"].startswith("int4_g") else 0


def _row_bytes(case):
    """Bytes of one token's K (or V) rows of all heads in the pool."""
    if _group(case):
        return case["k_heads"] * (case["dim"] // 2 + 4 * (case["dim"] // _group(case)))
    return case["k_heads"] * case["dim"] * (1 if case["kv"] == "e4m3" else 2)


def _lengths(case):
    """(rows, keys) of each request: the case's, whatever the seed."""
    mix, n = np.random.default_rng(case["mix"]), case["batch"]
    if case["op"] == "read":
        keys = mix.integers(case["len_lo"], case["len_hi"], size=n, endpoint=True)
        return keys, keys
    new = mix.integers(case["new_lo"], case["new_hi"], size=n, endpoint=True)
    if case["op"] == "attend":
        keys = mix.integers(case["kv_lo"], case["kv_hi"], size=n, endpoint=True)
        return new, np.maximum(keys, new)
    return new, new + mix.integers(1, case["prefix_hi"], size=n, endpoint=True)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _quantised(x, group):
    """Codes, steps and origins of groups of the last axis: the step is a 15th of the
    group's range and the origin its least value, both rounded to bf16."""
    g = x.float().unflatten(-1, (-1, group))
    lo, hi = g.amin(-1), g.amax(-1)
    # divided by a tensor: a scalar's reciprocal would break ties otherwise
    step = ((hi - lo) / torch.full_like(lo, 15.0)).to(torch.bfloat16).float()
    origin = lo.to(torch.bfloat16).float()
    at = (g - origin[..., None]) / torch.where(step > 0, step, 1.0)[..., None]
    code = at.round().clamp(0, 15).to(torch.uint8) * (step > 0)[..., None]
    return code.flatten(-2), step, origin


def _packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _words(step, origin):
    """[..., G, 4] bytes of the groups' words."""
    w = torch.stack([step.to(torch.bfloat16), origin.to(torch.bfloat16)], -1)
    return w.view(torch.uint8)


def _parts(case, pool):
    """Views of a 4-bit pool [pages, bytes]: codes and words by [page, slot, head]."""
    P, hk, d, g = case["page"], case["k_heads"], case["dim"], _group(case)
    n = P * hk * d // 2
    shape = (P, hk) if case["layout"] == "NHD" else (hk, P)
    code = pool[:, :n].unflatten(-1, shape + (d // 2,))
    words = pool[:, n:n + P * hk * (d // g) * 4].unflatten(-1, shape + (d // g, 4))
    if case["layout"] == "HND":
        code, words = code.transpose(1, 2), words.transpose(1, 2)
    return code, words


def _pool(g, case, pages):
    """K and V pools in one allocation [pages, 2, ...], every slot with a quantised row:
    channels of K spread unevenly, V alike."""
    P, hk, d, group = case["page"], case["k_heads"], case["dim"], _group(case)
    if not group:
        page = ((P, hk) if case["layout"] == "NHD" else (hk, P)) + (d,)
        if case["kv"] == "bf16":
            return torch.empty((pages, 2) + page, device=DEV,
                               dtype=torch.bfloat16).normal_(generator=g)
        codes = torch.randint(0, 127, (pages, 2) + page, generator=g, device=DEV,
                              dtype=torch.uint8)
        return codes | (torch.randint(0, 2, codes.shape, generator=g, device=DEV,
                                      dtype=torch.uint8) << 7)
    size = -(-P * _row_bytes(case) // 16) * 16
    kv = torch.zeros((pages, 2, size), device=DEV, dtype=torch.uint8)
    for i in range(2):
        x = torch.empty((pages, P, hk, d), device=DEV).normal_(generator=g)
        if i == 0:
            x *= torch.exp(0.5 * _normal(g, hk, d))
        code, step, origin = _quantised(x, group)
        c, w = _parts(case, kv[:, i])
        c.copy_(_packed(code))
        w.copy_(_words(step, origin))
    return kv


def _frequencies(case):
    """Radians a position for each pair of a head, as 64-bit numbers on the device."""
    s = ROPE_SCALING[case["scaling"]]
    half = case["rotary"] // 2
    f = s["base"] ** (torch.arange(half, dtype=torch.float64) * (-2.0 / case["rotary"]))
    if case["scaling"] == "linear":
        f = f / s["factor"]
    if case["scaling"] == "parts":
        turns = f * (s["original_len"] / (2 * math.pi))
        lo, hi = s["low_rotations"], s["high_rotations"]
        keep = ((turns - lo) / (hi - lo)).clamp(0, 1)
        f = f / s["factor"] * (1 - keep) + f * keep
    return f.to(DEV)


def _own_params(case):
    import paged_kv_attention_plan_gb300 as pka
    scales = SCALES.get(case["kv"], (1.0, 1.0))
    return pka.make_params(case["q_heads"], case["k_heads"], case["dim"], case["page"],
                           case["layout"], kv_dtype=case["kv"], k_scale=scales[0],
                           v_scale=scales[1])


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    P, hq, hk, d = case["page"], case["q_heads"], case["k_heads"], case["dim"]
    new, keys = _lengths(case)
    pages = -(-keys // P)
    indptr = np.concatenate([[0], np.cumsum(pages)])
    rows_at = np.concatenate([[0], np.cumsum(new)])
    pool = int(indptr[-1]) + int(indptr[-1]) // 8 + 1
    kv = _pool(g, case, pool)
    s = dict(case=case, rows=int(rows_at[-1]), most_rows=int(new.max()), most_keys=int(keys.max()),
             row_indptr=_i32(rows_at), kv_indptr=_i32(indptr),
             kv_indices=_i32(rng.permutation(pool)[: indptr[-1]]),
             last=_i32(keys - (pages - 1) * P), kv=kv)
    bf16, n = torch.bfloat16, s["rows"] + case.get("pad", 0)
    if case["op"] == "attend":
        s.update(q=_normal(g, n, hq, d).to(bf16), new=_i32(new), keys=_i32(keys),
                 out=torch.zeros((n, hq, d), device=DEV, dtype=bf16),
                 lse=torch.zeros((n, hq), device=DEV))
    else:
        s.update(k_out=torch.zeros((n, hk, d), device=DEV, dtype=bf16),
                 v_out=torch.zeros((n, hk, d), device=DEV, dtype=bf16),
                 begin=_i32(keys - new))
    if case["op"] == "append":
        s.update(k=_normal(g, n, hk, d).to(bf16), v=_normal(g, n, hk, d).to(bf16))
    if case["op"] == "rope_append":
        # bell-shaped rows of unit variance without far tails, as normalised heads have
        def rows(*shape):
            x = torch.rand(shape, generator=g, device=DEV) - torch.rand(shape, generator=g,
                                                                         device=DEV)
            return (x * math.sqrt(6.0)).to(bf16)
        if case["fused"]:
            x = rows(max(n, 1), hq + 2 * hk, d)[:n]
            q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        else:
            q, k, v = rows(n, hq, d), rows(n, hk, d), rows(n, hk, d)
        s.update(q=q, k=k, v=v, q_out=torch.zeros((n, hq, d), device=DEV, dtype=bf16),
                 f=_frequencies(case))
    if own:
        import paged_kv_attention_plan_gb300 as pka
        s["params"] = _own_params(case)
        if case["op"] == "rope_append":
            s["rope"] = pka.make_rope(case["rotary"], interleaved=case["interleaved"],
                                      **ROPE_SCALING[case["scaling"]])
        if case["op"] == "attend":
            s["attn"] = pka.BatchAttention()
            s["attn"].plan(rows_at.astype(np.int32), indptr.astype(np.int32),
                           (keys - (pages - 1) * P).astype(np.int32), num_qo_heads=hq,
                           num_kv_heads=hk, head_dim=d, page_size=P, layout=case["layout"],
                           mask_mode="causal", kv_dtype=case["kv"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


def _slots_of_rows(s):
    """Logical position, page and slot of each row of the batch, which are the last of its
    request's."""
    page = s["case"]["page"]
    row = torch.arange(s["rows"], device=DEV, dtype=torch.int32)
    r = torch.searchsorted(s["row_indptr"], row, right=True) - 1
    pages = s["kv_indptr"][r + 1] - s["kv_indptr"][r]
    end = (pages - 1) * page + s["last"][r]
    pos = end - s["row_indptr"][r + 1] + row
    return pos, s["kv_indices"][s["kv_indptr"][r] + pos // page].long(), (pos % page).long()


def _values(case, pool, page, slot, scale=1.0):
    """The rows [..., Hk, D] of the given pages and slots, in 32 bits."""
    if not _group(case):
        x = pool.view(torch.float8_e4m3fn) if case["kv"] == "e4m3" else pool
        x = x if case["layout"] == "NHD" else x.transpose(1, 2)
        return x[page, slot].float() * scale
    code, words = _parts(case, pool)
    c, w = code[page, slot], words[page, slot].view(torch.bfloat16).float()
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2).unflatten(-1, (-1, _group(case))).float()
    return (w[..., 1:] + w[..., :1] * c).flatten(-2)


def _store(case, pool, page, slot, x):
    code, step, origin = _quantised(x, _group(case))
    c, w = _parts(case, pool)
    c[page, slot] = _packed(code)
    w[page, slot] = _words(step, origin)


def _read(s, page, slot):
    ks, vs = SCALES.get(s["case"]["kv"], (1.0, 1.0))
    n, case = s["rows"], s["case"]
    s["k_out"][:n] = _values(case, s["kv"][:, 0], page, slot, ks).to(torch.bfloat16)
    s["v_out"][:n] = _values(case, s["kv"][:, 1], page, slot, vs).to(torch.bfloat16)
    return dict(k=s["k_out"], v=s["v_out"])


def _own_read(s):
    import paged_kv_attention_plan_gb300 as pka
    k, v = s["kv"][:, 0], s["kv"][:, 1]
    pka.pka_read_paged_kv_cache(s["params"], s["begin"], s["row_indptr"], s["kv_indptr"],
                                s["kv_indices"], s["last"], k, v, k.stride(0), s["k_out"],
                                s["v_out"])
    return dict(k=s["k_out"], v=s["v_out"])


def _plain_read(s):
    _, page, slot = _slots_of_rows(s)
    return _read(s, page, slot)


def _plain_append(s):
    _, page, slot = _slots_of_rows(s)
    _store(s["case"], s["kv"][:, 0], page, slot, s["k"])
    _store(s["case"], s["kv"][:, 1], page, slot, s["v"])
    return _read(s, page, slot)


def _own_append(s):
    import paged_kv_attention_plan_gb300 as pka
    k, v = s["kv"][:, 0], s["kv"][:, 1]
    pka.pka_append_paged_kv_cache(s["params"], s["k"], s["v"], s["row_indptr"], s["kv_indptr"],
                                  s["kv_indices"], s["last"], k, v, k.stride(0))
    return _own_read(s)


def _rotate(x, positions, f, case):
    """x [rows, heads, dim] rotated in 32 bits, the angles in 64."""
    rd = case["rotary"]
    angle = positions.double()[:, None, None] * f
    m = ROPE_SCALING[case["scaling"]].get("magnitude", 1.0)
    c, s = (torch.cos(angle) * m).float(), (torch.sin(angle) * m).float()
    x = x.float()
    head = x[..., :rd]
    if case["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    else:
        a, b = head[..., :rd // 2], head[..., rd // 2:]
        y = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    return torch.cat([y, x[..., rd:]], dim=-1)


def _plain_rope_append(s):
    case, n = s["case"], s["rows"]
    pos, page, slot = _slots_of_rows(s)
    s["q_out"][:n] = _rotate(s["q"][:n], pos, s["f"], case).to(torch.bfloat16)
    _store(case, s["kv"][:, 0], page, slot, _rotate(s["k"][:n], pos, s["f"], case))
    _store(case, s["kv"][:, 1], page, slot, s["v"][:n])
    return dict(_read(s, page, slot), q=s["q_out"])


def _own_rope_append(s):
    import paged_kv_attention_plan_gb300 as pka
    k, v = s["kv"][:, 0], s["kv"][:, 1]
    pka.pka_rope_append_paged_kv_cache(s["params"], s["rope"], s["q"], s["q_out"], s["k"], s["v"],
                                       s["row_indptr"], s["kv_indptr"], s["kv_indices"],
                                       s["last"], k, v, k.stride(0))
    return dict(_own_read(s), q=s["q_out"])


def _plain_attend(s):
    case = s["case"]
    d, hk, g = case["dim"], case["k_heads"], case["q_heads"] // case["k_heads"]
    # keys and rows of every request, padded to the longest
    j = torch.arange(s["most_keys"], device=DEV, dtype=torch.int32)
    there = j < s["keys"][:, None]
    at = torch.where(there, s["kv_indptr"][:-1, None] + j // case["page"], 0)
    page, slot = s["kv_indices"][at].long(), (j % case["page"]).long().expand(at.shape)
    k = _values(case, s["kv"][:, 0], page, slot).permute(0, 2, 3, 1)  # [batch, Hk, D, keys]
    v = _values(case, s["kv"][:, 1], page, slot).transpose(1, 2)      # [batch, Hk, keys, D]
    i = torch.arange(s["most_rows"], device=DEV, dtype=torch.int32)
    held = i < s["new"][:, None]
    row = torch.where(held, s["row_indptr"][:-1, None] + i, 0).long()
    q = s["q"][row].float().unflatten(2, (hk, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = (q @ k) * (1.0 / math.sqrt(d))                            # [batch, Hk, rows * g, keys]
    seen = j <= (s["keys"] - s["new"])[:, None, None] + i[:, None]    # [batch, rows, keys]
    seen = (seen & there[:, None]).repeat_interleave(g, 1)[:, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    o = (e @ v) / total
    lse = (top + torch.log(total)) / math.log(2.0)
    o = o.unflatten(2, (-1, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [batch, rows, Hq, D]
    lse = lse[..., 0].unflatten(2, (-1, g)).permute(0, 2, 1, 3).flatten(2, 3)
    s["out"].copy_(o[held].to(torch.bfloat16))
    s["lse"].copy_(lse[held])
    return _attended(s)


def _attended(s):
    # the statistics of decode rows are read by merges of their own; prompts' rows
    # have no reader for them
    if s["case"]["new_hi"] > 1:
        return dict(o=s["out"])
    return dict(o=s["out"], lse=s["lse"])


def _own_attend(s):
    lse = s["lse"] if s["case"]["new_hi"] == 1 else None
    s["attn"].run(s["q"], s["kv"][:, 0], s["kv"][:, 1], s["kv_indices"], out=s["out"], lse=lse,
                  return_lse=lse is not None)
    return _attended(s)


PLAIN = dict(append=_plain_append, rope_append=_plain_rope_append, read=_plain_read,
             attend=_plain_attend)
OWN = dict(append=_own_append, rope_append=_own_rope_append, read=_own_read, attend=_own_attend)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    new, keys = _lengths(case)
    rows, hq, hk, d = int(new.sum()), case["q_heads"], case["k_heads"], case["dim"]
    cached, plain = 2 * _row_bytes(case), 2 * hk * d * 2  # bytes of a token's K and V
    if case["op"] == "read":
        return dict(bytes=rows * (cached + plain), flops=0)
    if case["op"] == "attend":
        pairs = int((new * keys - new * (new - 1) // 2).sum())
        lse = 4 * hq * rows if case["new_hi"] == 1 else 0
        return dict(bytes=int(keys.sum()) * cached + rows * hq * d * 4 + lse,
                    flops=4 * d * hq * pairs)
    # rows in, into the pool, and out again
    move = rows * (plain + cached + plain)
    turned = rows * (hq + hk) * case.get("rotary", 0) * 3
    return dict(bytes=max(1, move + (rows * hq * d * 4 if case["op"] == "rope_append" else 0)),
                flops=turned + rows * 2 * hk * d * 4)


# ---------------------------------------------------------------------------
# The outputs from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _bf16_of(x):
    """64-bit numbers rounded to the nearest bf16: 7 of the 52 bits of the fraction stay,
    ties to even."""
    b = x.contiguous().view(torch.int64)
    return ((b + ((1 << 44) - 1) + ((b >> 45) & 1)) & -(1 << 45)).view(torch.float64)


def _kept(x, group):
    """What 4 bits keep of 64-bit numbers."""
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // group, group))
    least, range_ = y.min(-1, keepdim=True)[0], y.max(-1, keepdim=True)[0]
    step, origin = _bf16_of((range_ - least) / torch.full_like(least, 15.0)), _bf16_of(least)
    n = torch.clamp(torch.round((y - origin) / step), 0, 15)
    return torch.where(step > 0, origin + step * n, origin.expand(y.shape)).reshape(x.shape)


def _held(case, kv, pages, slots):
    """The rows [n, Hk, D] of a pool in 64 bits, byte by byte."""
    P, hk, d, g = case["page"], case["k_heads"], case["dim"], _group(case)
    head = torch.arange(hk, device=DEV)
    at = slots[:, None] * hk + head if case["layout"] == "NHD" else head * P + slots[:, None]
    if not g:
        flat = kv.reshape(kv.shape[0], P * hk, d)[pages[:, None], at]
        return (flat.view(torch.float8_e4m3fn) if case["kv"] == "e4m3" else flat).double()
    byte = at[..., None] * (d // 2) + torch.arange(d, device=DEV) // 2
    code = kv[pages[:, None, None], byte].long()
    code = torch.where(torch.arange(d, device=DEV) % 2 == 1, code // 16, code % 16)
    word = P * hk * d // 2 + 4 * (at[..., None] * (d // g) + torch.arange(d, device=DEV) // g)

    def half(first):  # a bf16 number from its two bytes
        b = [kv[pages[:, None, None], word + first + i].to(torch.int32) for i in range(2)]
        return ((b[0] + 256 * b[1]) << 16).view(torch.float32).double()
    return half(2) + half(0) * code


def _turned(x, pos, case):
    """x times exp(i * angle) pair by pair, in complex numbers of 64-bit parts."""
    s, rd = ROPE_SCALING[case["scaling"]], case["rotary"]
    f = np.array([s["base"] ** (-2.0 * i / rd) for i in range(rd // 2)])
    if case["scaling"] == "linear":
        f = f / s["factor"]
    if case["scaling"] == "parts":
        per = s["original_len"] * f / (2 * np.pi)
        lo, hi = s["low_rotations"], s["high_rotations"]
        w = np.where(per <= lo, 0.0, np.where(per >= hi, 1.0, (per - lo) / (hi - lo)))
        f = w * f + (1 - w) * f / s["factor"]
    angle = torch.outer(pos.double(), torch.from_numpy(f).to(DEV))
    turn = torch.polar(torch.full_like(angle, s.get("magnitude", 1.0)), angle)[:, None]
    y = x.double().clone()
    first = slice(0, rd, 2) if case["interleaved"] else slice(0, rd // 2)
    second = slice(1, rd, 2) if case["interleaved"] else slice(rd // 2, rd)
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    rows_at, ptr, ids, last = (s[n].cpu().numpy().astype(np.int64) for n in
                               ("row_indptr", "kv_indptr", "kv_indices", "last"))
    P, n = case["page"], case["batch"]
    count = np.diff(rows_at)
    end = (np.diff(ptr) - 1) * P + last
    if case["op"] in ("append", "rope_append"):
        pos = np.concatenate([np.arange(end[r] - count[r], end[r]) for r in range(n)])
        out = {x: s[x + "_out"].double() for x in "kv"}
        m, x = s["rows"], s["k"][: s["rows"]].double()
        if case["op"] == "rope_append":
            pos = torch.from_numpy(pos).to(DEV)
            x = _turned(x, pos, case)
            out["q"] = s["q_out"].double()
            out["q"][:m] = _turned(s["q"][:m], pos, case)
        out["k"][:m] = _kept(x, _group(case))
        out["v"][:m] = _kept(s["v"][:m].double(), _group(case))
        return out
    # request by request: which pages and slots its keys lie in
    where = []
    for r in range(n):
        j = np.arange(end[r])
        where.append(tuple(torch.from_numpy(a).to(DEV) for a in (ids[ptr[r] + j // P], j % P)))
    if case["op"] == "read":
        scale = SCALES.get(case["kv"], (1.0, 1.0))
        return {x: torch.cat([_held(case, s["kv"][:, i], *w) for w in where]) * scale[i]
                for i, x in enumerate("kv")}
    g, o, lse = case["q_heads"] // case["k_heads"], [], []
    if float((count * end).sum()) * case["q_heads"] * case["dim"] > 2e12:
        return None
    for r, w in enumerate(where):
        k, v = (_held(case, s["kv"][:, i], *w) for i in range(2))
        hidden = torch.arange(end[r], device=DEV)[None] > \
            torch.arange(count[r], device=DEV)[:, None] + (end[r] - count[r])
        q = s["q"][rows_at[r]:rows_at[r + 1]].double()
        heads = []
        for h in range(case["q_heads"]):
            score = (q[:, h] @ k[:, h // g].T) / math.sqrt(case["dim"])
            score = score.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(score, -1)
            heads.append((torch.exp(score - z[:, None]) @ v[:, h // g], z / math.log(2.0)))
        o.append(torch.stack([x[0] for x in heads], 1))
        lse.append(torch.stack([x[1] for x in heads], 1))
    out = dict(o=torch.cat(o))
    if case["new_hi"] == 1:
        out["lse"] = torch.cat(lse)
    return out
