"""Measured cases of the operators around the paged KV cache: rotary
positions, the append that rotates, and the copying, forking, compacting,
taking and returning of pages.

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, through the library's entry points.  ``exact`` gives the floating
outputs in 64 bits, written apart from both.
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
        # one decode step of the benchmark's 64 requests: q and k as slices of the
        # projection's output row, histories up to 128K tokens
        dict(name="rope decode 64", op="rope", rows=64, q_heads=32, k_heads=8, dim=128,
             rotary=128, interleaved=False, transpose=False, scaling="none", fused=True,
             max_pos=131072),
        # the gradient of a training batch's rotation: many rows, as many kv as qo
        # heads, a quarter of each head rotated, neighbouring pairs
        dict(name="rope gradient 16387", op="rope", rows=16387, q_heads=32, k_heads=32, dim=128,
             rotary=32, interleaved=True, transpose=True, scaling="linear", fused=False,
             max_pos=32768),
        # a decode step into 8-bit pools
        dict(name="rope_append decode e4m3", op="rope_append", batch=256, new_lo=1, new_hi=1,
             prefix_hi=1000, mix=1, pad=0, page=16, layout="HND", kv="e4m3", q_heads=32, k_heads=8,
             dim=128, rotary=128, interleaved=False, scaling="parts", fused=True),
        # the benchmark's append-prefill step (16 requests of 128..1024 new rows), as a
        # captured step sees it: the buffers end in rows of no request
        dict(name="rope_append prefill", op="rope_append", batch=16, new_lo=128, new_hi=1024,
             prefix_hi=4096, mix=2, pad=61, page=16, layout="NHD", kv="bf16", q_heads=32, k_heads=8,
             dim=128, rotary=128, interleaved=False, scaling="parts", fused=True),
        # the partly filled last pages of eight samples of one prompt, eight layers
        dict(name="copy 8 partial pages", op="copy", layers=8, pages=512, copies=8, partial=True,
             page=16, layout="NHD", kv="bf16", k_heads=8, dim=128),
        # pages moved by a large defragmentation, four layers in one allocation
        dict(name="copy 4001 pages", op="copy", layers=4, pages=8192, copies=4001, partial=False,
             page=16, layout="HND", kv="bf16", k_heads=8, dim=128),
        # eight samples of one 2,040-token prompt, each with room for its next page,
        # then their return
        dict(name="fork 1 into 8", op="fork", parents=1, len_lo=2040, len_hi=2040, children=8,
             mix=3, grow=1, pages=1024, page=16, layers=8, layout="NHD", kv="bf16", k_heads=8,
             dim=128),
        # a step of beam search over a token pool (page size 1): 256 beams from 64
        dict(name="fork 64 into 256", op="fork", parents=64, len_lo=1024, len_hi=6144,
             children=256, mix=4, grow=1, pages=1000003, page=1, layers=0, layout="NHD", kv="bf16",
             k_heads=8, dim=128),
        # a small cache after requests came and went
        dict(name="compact 2048", op="compact", pages=2048, live=0.6, requests=33, page=16,
             layers=1, layout="NHD", kv="bf16", k_heads=8, dim=128),
        # a token pool of 8-bit rows
        dict(name="compact 500009", op="compact", pages=500009, live=0.5, requests=200, page=1,
             layers=1, layout="HND", kv="e4m3", k_heads=8, dim=128),
        # the pages that a decode step's requests grow into, and their return
        dict(name="pages 64 of 8192", op="pages", pages=8192, live=0.7, take=64),
        # a long prompt's slots in a token pool, and their return
        dict(name="pages 131072 of 1.5M", op="pages", pages=1500007, live=0.8, take=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_append", "copy", "fork", "compact", "pages"])
    dim = rng.choice([64, 128])
    q_heads, k_heads = rng.choice([(8, 1), (8, 2), (32, 8), (32, 32), (28, 7), (5, 5), (64, 8)])
    rotary = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])
    shape = dict(interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "parts"]),
                 fused=rng.random() < 0.5)
    kv = dict(page=rng.choice([1, 3, 4, 16, 64]), layout=rng.choice(["NHD", "HND"]),
              kv=rng.choice(["bf16", "e4m3"]), dim=dim)
    if op == "rope":
        rows = min(_log(rng, 1, 16387), 16387 * 64 * 128 // ((q_heads + k_heads) * dim))
        return dict(op=op, rows=rows, q_heads=q_heads, k_heads=k_heads, dim=dim, rotary=rotary,
                    transpose=rng.random() < 0.5, max_pos=_log(rng, 100, 2000000), **shape)
    if op == "rope_append":
        batch = _log(rng, 1, 256)
        new_hi = 1 if rng.random() < 0.5 else max(1, _log(rng, 1, 9000) // batch)
        return dict(op=op, batch=batch, new_lo=min(new_hi, rng.randint(0, 2)), new_hi=new_hi,
                    prefix_hi=min(_log(rng, 16, 4096), 100000 // batch),
                    mix=rng.randint(0, 1 << 30),
                    pad=rng.choice([0, 0, rng.randint(1, 64)]), q_heads=q_heads, k_heads=k_heads,
                    rotary=rotary, **kv, **shape)
    token = 4 * k_heads * dim  # bytes of one token's K and V rows in bf16
    if op == "copy":
        layers = rng.randint(1, 8)
        pages = max(8, min(_log(rng, 32, 16384), (1 << 31) // (token * kv["page"] * layers)))
        return dict(op=op, layers=layers, pages=pages, copies=max(1, _log(rng, 1, pages // 2) - 1),
                    partial=rng.random() < 0.5, k_heads=k_heads, **kv)
    if op == "fork":
        parents = _log(rng, 1, 64)
        len_hi = _log(rng, 40, 6144)
        children = _log(rng, 1, 256)
        pages = parents * (len_hi // kv["page"] + 1) + 3 * children + rng.randint(1, 5000)
        layers = min(rng.randint(0, 4), (1 << 30) // (pages * token * kv["page"]))
        return dict(op=op, parents=parents, len_lo=rng.randint(1, len_hi), len_hi=len_hi,
                    children=children, mix=rng.randint(0, 1 << 30), grow=rng.randint(0, 2),
                    pages=pages, layers=layers, k_heads=k_heads, **kv)
    if op == "compact":
        pages = max(16, min(_log(rng, 64, 500000), (1 << 29) // (token * kv["page"])))
        return dict(op=op, pages=pages, live=round(rng.uniform(0.05, 0.95), 3),
                    requests=rng.randint(1, 200), layers=1, k_heads=k_heads, **kv)
    pages = _log(rng, 64, 1500007)
    live = round(rng.uniform(0.0, 0.9), 3)
    take = _log(rng, 1, max(2, min(131072, int(pages * (1 - live)) // 2)))
    return dict(op=op, pages=pages, live=live, take=take)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

ROPE_SCALING = {
    "none": dict(base=10000.0),
    # positions of a context four times as long as the trained one, divided by four
    "linear": dict(base=10000.0, scaling="linear", factor=4.0),
    # slow pairs divided by eight, fast ones kept, a ramp between 1 and 32 turns over
    # the trained 8,192 positions, and the magnitude that goes with it
    "parts": dict(base=500000.0, scaling="parts", factor=8.0, original_len=8192.0,
                  low_rotations=1.0, high_rotations=32.0,
                  magnitude=0.1 * math.log(8.0) + 1.0),
}


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


def _own_rope(case):
    import paged_kv_attention_plan_gb300 as pka
    return pka.make_rope(case["rotary"], interleaved=case["interleaved"],
                         **ROPE_SCALING[case["scaling"]])


def _own_params(case):
    import paged_kv_attention_plan_gb300 as pka
    scales = SCALES[case["kv"]]
    return pka.make_params(case.get("q_heads", case["k_heads"]), case["k_heads"], case["dim"],
                           case["page"], case["layout"], kv_dtype=case["kv"], k_scale=scales[0],
                           v_scale=scales[1])


# the scales of 8-bit K and V: rotated rows have the spread of the unrotated ones
SCALES = {"bf16": (1.0, 1.0), "e4m3": (0.03125, 0.02)}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _pool(g, case, layers, pages):
    """K and V of all layers in one allocation [layers, pages, 2, ...]: bf16 values or e4m3 codes."""
    page = ((case["page"], case["k_heads"]) if case["layout"] == "NHD" else
            (case["k_heads"], case["page"])) + (case["dim"],)
    shape = (layers, pages, 2) + page
    if case["kv"] == "e4m3":
        codes = torch.randint(0, 127, shape, generator=g, device=DEV, dtype=torch.uint8)
        sign = torch.randint(0, 2, shape, generator=g, device=DEV, dtype=torch.uint8)
        return codes | (sign << 7)
    return torch.empty(shape, device=DEV, dtype=torch.bfloat16).normal_(generator=g)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tables(rng, lengths, page, ids):
    """CSR page table of requests of the given lengths whose pages are the given ids in order."""
    pages = -(-lengths // page)
    indptr = np.concatenate([[0], np.cumsum(pages)])
    last = np.where(pages > 0, lengths - (pages - 1) * page, 1)
    return indptr, ids[: indptr[-1]], last


# The lengths of a batch go by the case's ``mix``, so that its outputs have one shape; page
# ids and payloads go by the seed.

def _rows(g, case, rows):
    """q, k and v rows of a step: slices of one projection output, or tensors of their own."""
    hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
    if case["fused"]:
        x = _normal(g, rows, hq + 2 * hk, d)
        return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    return _normal(g, rows, hq, d), _normal(g, rows, hk, d), _normal(g, rows, hk, d)


def prepare(case, seed):
    return PREPARE[case["op"]](case, seed)


def _prepare_rope(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    q, k, _ = _rows(g, case, case["rows"])
    s = dict(case=case, q=q, k=k, f=_frequencies(case),
             positions=_i32(rng.integers(0, case["max_pos"], case["rows"])),
             q_out=torch.empty(q.shape, dtype=q.dtype, device=DEV),
             k_out=torch.empty(k.shape, dtype=k.dtype, device=DEV))
    if own:
        s["rope"] = _own_rope(case)
    return s


def _prepare_rope_append(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, mix = case["batch"], np.random.default_rng(case["mix"])
    new = mix.integers(case["new_lo"], case["new_hi"], size=n, endpoint=True)
    total = new + mix.integers(1, case["prefix_hi"], size=n, endpoint=True)
    pages = int((-(-total // case["page"])).sum())
    pool = pages + pages // 8 + 1
    indptr, indices, last = _tables(rng, total, case["page"], rng.permutation(pool))
    rows = int(new.sum()) + case["pad"]
    q, k, v = _rows(g, case, max(rows, 1))
    kv = _pool(g, case, 1, pool)[0]
    s = dict(case=case, q=q, k=k, v=v, q_out=torch.zeros(q.shape, dtype=q.dtype, device=DEV),
             append_indptr=_i32(np.concatenate([[0], np.cumsum(new)])), kv_indptr=_i32(indptr),
             kv_indices=_i32(indices), last=_i32(last), kv=kv, rows=int(new.sum()),
             f=_frequencies(case))
    if own:
        s["rope"], s["params"] = _own_rope(case), _own_params(case)
    return s


def _prepare_copy(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    ids = rng.permutation(case["pages"])
    n = case["copies"]
    s = dict(case=case, kv=_pool(g, case, case["layers"], case["pages"]), src=_i32(ids[:n]),
             dst=_i32(ids[n:2 * n]), slots=None)
    if case["partial"]:
        s["slots"] = _i32(rng.integers(1, case["page"], size=n, endpoint=True))
    if own:
        s["params"] = _own_params(case)
    return s


def _prepare_fork(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    P, n, c = case["page"], case["parents"], case["children"]
    mix = np.random.default_rng(case["mix"])
    lengths = mix.integers(case["len_lo"], case["len_hi"], size=n, endpoint=True)
    indptr, indices, last = _tables(rng, lengths, P, rng.permutation(case["pages"]))
    parent = mix.integers(0, n, size=c)
    pages = indptr[1:] - indptr[:-1]
    child = np.concatenate([[0], np.cumsum(pages[parent] + case["grow"])])
    shared = pages - (last < P)
    refs = np.zeros(case["pages"], np.int64)
    refs[indices] = 1
    s = dict(case=case, refs=_i32(refs), kv_indptr=_i32(indptr), kv_indices=_i32(indices),
             last=_i32(last), parent=_i32(parent), child_indptr=_i32(child),
             child_indices=torch.full((int(child[-1]),), -1, dtype=torch.int32, device=DEV),
             src=torch.full((c,), -1, dtype=torch.int32, device=DEV),
             dst=torch.full((c,), -1, dtype=torch.int32, device=DEV),
             slots=torch.full((c,), -1, dtype=torch.int32, device=DEV),
             counts=torch.zeros(2, dtype=torch.int32, device=DEV),
             fresh=int(child[-1] - shared[parent].sum()), copies=int((last[parent] < P).sum()),
             kv=_pool(g, case, case["layers"], case["pages"]) if case["layers"] else None)
    if own:
        s["params"] = _own_params(case)
    return s


def _prepare_compact(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n = case["pages"]
    live = max(1, int(n * case["live"]))
    ids = rng.permutation(n)[:live]
    # each request: pages of its own and the first pages of the pool's shared prompt
    prompt = ids[: max(1, live // 100)]
    own_ids = ids[len(prompt):]
    cuts = np.sort(rng.integers(0, len(own_ids) + 1, size=case["requests"] - 1))
    parts = np.split(own_ids, cuts)
    indices = np.concatenate([np.concatenate([prompt[: max(1, 2000 // case["requests"])], p])
                              for p in parts] + [prompt])
    refs = np.bincount(indices, minlength=n)
    s = dict(case=case, refs=_i32(refs), kv_indices=_i32(indices),
             refs_out=torch.full((n,), -1, dtype=torch.int32, device=DEV),
             indices_out=torch.full((len(indices),), -1, dtype=torch.int32, device=DEV),
             map=torch.full((n,), -2, dtype=torch.int32, device=DEV),
             src=torch.full((n // 2,), -1, dtype=torch.int32, device=DEV),
             dst=torch.full((n // 2,), -1, dtype=torch.int32, device=DEV),
             counts=torch.zeros(2, dtype=torch.int32, device=DEV),
             kv=_pool(g, case, case["layers"], n))
    if own:
        s["params"] = _own_params(case)
    return s


def _prepare_pages(case, seed):
    rng = np.random.default_rng(seed)
    n = case["pages"]
    refs = np.zeros(n, np.int64)
    held = rng.permutation(n)[: int(n * case["live"])]
    refs[held] = rng.integers(1, 4, size=len(held))
    return dict(case=case, refs=_i32(refs),
                pages=torch.full((case["take"],), -1, dtype=torch.int32, device=DEV))


PREPARE = dict(rope=_prepare_rope, rope_append=_prepare_rope_append, copy=_prepare_copy,
               fork=_prepare_fork, compact=_prepare_compact, pages=_prepare_pages)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


def _values(kv):
    """The pool's numbers: bf16, or e4m3 values (without the pool's scale)."""
    return kv.view(torch.float8_e4m3fn) if kv.dtype == torch.uint8 else kv


def _bits(kv):
    """The pool's bit patterns, for operators that only move them."""
    return kv if kv.dtype == torch.uint8 else kv.view(torch.int16)


def _rotate(x, positions, f, case, transpose=False):
    """x [rows, heads, dim] rotated in 32 bits, the angles in 64."""
    rd = case["rotary"]
    angle = positions.double()[:, None, None] * f
    m = ROPE_SCALING[case["scaling"]].get("magnitude", 1.0)
    c, s = (torch.cos(angle) * m).float(), (torch.sin(angle) * m).float()
    if transpose:
        s = -s
    x = x.float()
    head = x[..., :rd]
    if case["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    else:
        a, b = head[..., :rd // 2], head[..., rd // 2:]
        y = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    return torch.cat([y, x[..., rd:]], dim=-1)


def _plain_rope(s):
    case = s["case"]
    q = _rotate(s["q"], s["positions"], s["f"], case, case["transpose"])
    k = _rotate(s["k"], s["positions"], s["f"], case, case["transpose"])
    return dict(q=q.to(torch.bfloat16), k=k.to(torch.bfloat16))


def _own_rope_run(s):
    import paged_kv_attention_plan_gb300 as pka
    pka.pka_apply_rope(s["rope"], s["positions"], s["q"], s["q_out"], s["k"], s["k_out"],
                       transpose=s["case"]["transpose"])
    return dict(q=s["q_out"], k=s["k_out"])


def _slots_of_rows(s, page):
    """Logical position, page and slot of each appended row."""
    row = torch.arange(s["rows"], device=DEV, dtype=torch.int32)
    r = torch.searchsorted(s["append_indptr"], row, right=True) - 1
    pages = s["kv_indptr"][r + 1] - s["kv_indptr"][r]
    end = (pages - 1) * page + s["last"][r]
    pos = end - s["append_indptr"][r + 1] + row
    return pos, s["kv_indices"][s["kv_indptr"][r] + pos // page].long(), (pos % page).long()


def _plain_rope_append(s):
    case, n = s["case"], s["rows"]
    pos, page, slot = _slots_of_rows(s, case["page"])
    q = _rotate(s["q"][:n], pos, s["f"], case).to(torch.bfloat16)
    k = _rotate(s["k"][:n], pos, s["f"], case)
    v = s["v"][:n].float()
    s["q_out"][:n] = q
    if case["kv"] == "e4m3":
        ks, vs = SCALES["e4m3"]
        k = (k / ks).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / vs).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    if case["layout"] == "NHD":
        s["kv"][page, 0, slot] = k
        s["kv"][page, 1, slot] = v
    else:
        s["kv"][page, 0, :, slot] = k
        s["kv"][page, 1, :, slot] = v
    return dict(q=s["q_out"], k=_values(s["kv"][:, 0]), v=_values(s["kv"][:, 1]))


def _own_rope_append(s):
    import paged_kv_attention_plan_gb300 as pka
    k, v = s["kv"][:, 0], s["kv"][:, 1]
    pka.pka_rope_append_paged_kv_cache(s["params"], s["rope"], s["q"], s["q_out"], s["k"], s["v"],
                                       s["append_indptr"], s["kv_indptr"], s["kv_indices"],
                                       s["last"], k, v, k.stride(0))
    return dict(q=s["q_out"], k=_values(k), v=_values(v))


def _copy(kv, case, src, dst, slots):
    """Pages src of every layer's K and V written over pages dst: whole, or their first slots."""
    src, dst = src.long(), dst.long()
    new = kv[:, src]
    if slots is not None:
        keep = torch.arange(case["page"], device=DEV) < slots[:, None]
        shape = (1, len(src), 1, case["page"], 1, 1) if case["layout"] == "NHD" else \
            (1, len(src), 1, 1, case["page"], 1)
        new = torch.where(keep.view(shape), new, kv[:, dst])
    kv[:, dst] = new


def _plain_copy(s):
    _copy(s["kv"], s["case"], s["src"], s["dst"], s["slots"])
    return dict(kv=_bits(s["kv"]))


def _own_copy(s):
    import paged_kv_attention_plan_gb300 as pka
    pka.pka_copy_pages(s["params"], s["kv"][:, :, 0], s["kv"][:, :, 1], s["src"], s["dst"],
                       s["slots"])
    return dict(kv=_bits(s["kv"]))


def _lowest_free(refs, n):
    """The n lowest pages without a reference."""
    rank = torch.cumsum(refs == 0, 0, dtype=torch.int32)
    return torch.searchsorted(rank, torch.arange(1, n + 1, device=DEV, dtype=torch.int32),
                              out_int32=True)


def _plain_fork(s):
    case = s["case"]
    fresh = _lowest_free(s["refs"], s["fresh"])
    # the child, the place in its table and the parent of every entry
    entry = torch.arange(len(s["child_indices"]), device=DEV, dtype=torch.int32)
    child = torch.searchsorted(s["child_indptr"], entry, right=True) - 1
    place = entry - s["child_indptr"][child]
    first = s["kv_indptr"][s["parent"]]
    pages = s["kv_indptr"][s["parent"] + 1] - first
    partial = (s["last"][s["parent"]] < case["page"]) & (pages > 0)
    full = pages - partial.int()
    shared = place < full[child]
    nth = (torch.cumsum(~shared, 0) - 1).clamp(min=0)
    old = s["kv_indices"][(first[child] + place).clamp(max=len(s["kv_indices"]) - 1)]
    ids = old if s["fresh"] == 0 else torch.where(shared, old, fresh[nth.clamp(max=s["fresh"] - 1)])
    s["child_indices"].copy_(ids)
    s["refs"].index_add_(0, ids, torch.ones_like(ids))
    n = s["copies"]
    which = torch.searchsorted(torch.cumsum(partial, 0), torch.arange(1, n + 1, device=DEV))
    s["src"][:n] = s["kv_indices"][first[which] + full[which]]
    s["dst"][:n] = ids[s["child_indptr"][which] + full[which]]
    s["slots"][:n] = s["last"][s["parent"][which]]
    s["counts"][0], s["counts"][1] = n, s["fresh"]
    if s["kv"] is not None:
        _copy(s["kv"], case, s["src"][:n], s["dst"][:n], s["slots"][:n])
    out = _forked(s)
    s["refs"].index_add_(0, ids, torch.full_like(ids, -1))
    return out


def _forked(s):
    out = dict(child_indices=s["child_indices"], src=s["src"], dst=s["dst"], slots=s["slots"],
               counts=s["counts"], refs=s["refs"])
    if s["kv"] is not None:
        out["kv"] = _bits(s["kv"])
    return out


def _own_fork(s):
    import paged_kv_attention_plan_gb300 as pka
    pka.pka_fork_pages(s["case"]["page"], s["refs"], s["kv_indptr"], s["kv_indices"], s["last"],
                       s["parent"], s["child_indptr"], s["child_indices"], s["src"], s["dst"],
                       s["slots"], s["counts"])
    if s["kv"] is not None:
        pka.pka_copy_pages(s["params"], s["kv"][:, :, 0], s["kv"][:, :, 1], s["src"], s["dst"],
                           s["slots"], s["counts"])
    pka.pka_free_pages(s["refs"], s["child_indices"])
    return _forked(s)


def _plain_compact(s):
    refs, n = s["refs"], len(s["refs"])
    page = torch.arange(n, device=DEV, dtype=torch.int32)
    live = refs > 0
    up_to = torch.cumsum(live, 0, dtype=torch.int32)
    before, total = up_to - live.int(), up_to[-1]
    hole, mover = ~live & (page < total), live & (page >= total)
    place = torch.where(hole, page - before, total - 1 - before)
    cap = n // 2
    dst = torch.full((cap + 1,), -1, dtype=torch.int32, device=DEV)
    src = torch.full((cap + 1,), -1, dtype=torch.int32, device=DEV)
    dst.scatter_(0, torch.where(hole, place, cap).long(), page)
    src.scatter_(0, torch.where(mover, place, cap).long(), page)
    moves = int(mover.sum())  # the program reads it to size its copies
    s["src"][:moves], s["dst"][:moves] = src[:moves], dst[:moves]
    s["counts"][0], s["counts"][1] = moves, total
    to = torch.where(mover, dst[torch.where(mover, place, cap).long()], page)
    s["map"].copy_(torch.where(live, to, -1))
    s["indices_out"].copy_(to[s["kv_indices"]])
    s["refs_out"].zero_()
    s["refs_out"].scatter_add_(0, to.long(), torch.where(live, refs, 0))
    _copy(s["kv"], s["case"], s["src"][:moves], s["dst"][:moves], None)
    return _compacted(s)


def _compacted(s):
    return dict(refs=s["refs_out"], indices=s["indices_out"], map=s["map"], src=s["src"],
                dst=s["dst"], counts=s["counts"], kv=_bits(s["kv"]))


def _own_compact(s):
    import paged_kv_attention_plan_gb300 as pka
    pka.pka_compact_pages(s["refs"], s["kv_indices"], s["refs_out"], s["indices_out"], s["map"],
                          s["src"], s["dst"], s["counts"])
    pka.pka_copy_pages(s["params"], s["kv"][:, :, 0], s["kv"][:, :, 1], s["src"], s["dst"], None,
                       s["counts"])
    return _compacted(s)


def _plain_pages(s):
    pages = _lowest_free(s["refs"], s["case"]["take"])
    s["refs"].index_add_(0, pages, torch.ones_like(pages))
    s["pages"].copy_(pages)
    s["refs"].index_add_(0, s["pages"], torch.full_like(pages, -1))
    return dict(pages=s["pages"], refs=s["refs"])


def _own_pages(s):
    import paged_kv_attention_plan_gb300 as pka
    pka.pka_alloc_pages(s["refs"], s["pages"])
    pka.pka_free_pages(s["refs"], s["pages"])
    return dict(pages=s["pages"], refs=s["refs"])


PLAIN = dict(rope=_plain_rope, rope_append=_plain_rope_append, copy=_plain_copy,
             fork=_plain_fork, compact=_plain_compact, pages=_plain_pages)
OWN = dict(rope=_own_rope_run, rope_append=_own_rope_append, copy=_own_copy, fork=_own_fork,
           compact=_own_compact, pages=_own_pages)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope":
        heads = case["rows"] * (case["q_heads"] + case["k_heads"])
        return dict(bytes=heads * case["dim"] * 4 + 4 * case["rows"],
                    flops=heads * case["rotary"] * 3)
    if op == "pages":
        return dict(bytes=4 * case["pages"] + case["take"] * (4 + 4 + 4 + 8), flops=0)
    item = 1 if case["kv"] == "e4m3" else 2
    row = case["k_heads"] * case["dim"]  # elements of a token's K (or V)
    if op == "rope_append":
        rows = case["batch"] * (case["new_lo"] + case["new_hi"]) // 2
        return dict(bytes=max(1, rows * (case["q_heads"] * case["dim"] * 4 + row * (4 + 2 * item))),
                    flops=rows * (case["q_heads"] + case["k_heads"]) * case["rotary"] * 3)
    if op == "copy":
        slots = (case["page"] + 1) / 2 if case["partial"] else case["page"]
        return dict(bytes=case["layers"] * case["copies"] * 2 * slots * row * item * 2, flops=0)
    if op == "fork":
        pages = (case["len_lo"] + case["len_hi"]) / 2 / case["page"]
        entries = case["children"] * (pages + case["grow"])
        table = 4 * case["pages"] + min(case["parents"], case["children"]) * pages * (4 + 8 + 8)
        moved = (case["layers"] * case["children"] * (case["page"] - 1) / 2 * 2 * row * item * 2)
        return dict(bytes=table + entries * (4 + 4) + moved, flops=0)
    n, f = case["pages"], case["live"]
    moved = n * f * (1 - f)
    return dict(bytes=12 * n + 8 * n * f + moved * (8 + case["layers"] * 2 * case["page"] * row *
                                                    item * 2), flops=0)


# ---------------------------------------------------------------------------
# The floating outputs from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _turned(x, pos, case, sign):
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
    turn = torch.polar(torch.full_like(angle, s.get("magnitude", 1.0)), sign * angle)[:, None]
    y = x.double().clone()
    first = slice(0, rd, 2) if case["interleaved"] else slice(0, rd // 2)
    second = slice(1, rd, 2) if case["interleaved"] else slice(rd // 2, rd)
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    if case["op"] not in ("rope", "rope_append"):
        return None  # whole numbers and moved bits
    s = prepare(case, seed)
    if case["op"] == "rope":
        sign = -1.0 if case["transpose"] else 1.0
        return dict(q=_turned(s["q"], s["positions"], case, sign),
                    k=_turned(s["k"], s["positions"], case, sign))
    # row by row on the host: where each appended row goes
    app, ptr, ids, last = (s[n].cpu().numpy().astype(np.int64) for n in
                           ("append_indptr", "kv_indptr", "kv_indices", "last"))
    P, where = case["page"], []
    for r in range(case["batch"]):
        end = (ptr[r + 1] - ptr[r] - 1) * P + last[r]
        for t in range(app[r + 1] - app[r]):
            p = end - (app[r + 1] - app[r]) + t
            where.append((p, ids[ptr[r] + p // P], p % P))
    where = torch.tensor(where, dtype=torch.int64, device=DEV).reshape(-1, 3)
    pos, page, slot, n = where[:, 0], where[:, 1], where[:, 2], len(where)
    q = s["q_out"].double()
    q[:n] = _turned(s["q"][:n], pos, case, 1.0)
    k, v = _values(s["kv"][:, 0]).double(), _values(s["kv"][:, 1]).double()
    ks, vs = SCALES[case["kv"]]
    most = 448.0 if case["kv"] == "e4m3" else math.inf
    new_k = (_turned(s["k"][:n], pos, case, 1.0) / ks).clamp(-most, most)
    new_v = (s["v"][:n].double() / vs).clamp(-most, most)
    if case["layout"] == "HND":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    k[page, slot], v[page, slot] = new_k, new_v
    if case["layout"] == "HND":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return dict(q=q, k=k, v=v)
