"""The operators that fill and read a paged cache held in 4 bits, as cases to measure.

Three operators, in the order in which a step runs them:

``tables``  block tables built or grown on the GPU from the requests' lengths and a list of free pages, with the slot and
            the position of every new token.
``rope``    the norms of queries and keys for each head and their position rotation in one pass, the keys written to
            their cache slots, in the types that the cache holds.
``mla4``    the step's latent rows packed into a 4-bit cache, and the sparse attention over the selected rows of it.

``run`` computes a case in plain torch operations, or with the framework's kernels where ``own`` is true.
"""
import math

import torch

own = False

# latent rows of 416 bytes: 512 E2M1 codes (eight values to a 32-bit word: value 2j in its bits 4j .. 4j + 3, value 2j + 1 in
# 16 + 4j .. 19 + 4j), 32 scales (one per 16 values, unsigned, 5 bits of exponent and 3 of mantissa: code c is
# 2^(c//8 - 16) * (1 + c%8 / 8), but 0 is 0 and 255 is NaN), 64 bf16 rope values
ROW4 = 416
TO_NIBBLES, FROM_NIBBLES = (0, 2, 4, 6, 1, 3, 5, 7), (0, 4, 1, 5, 2, 6, 3, 7)
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SOFTMAX_SCALE = 1.0 / math.sqrt(576)


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # --- block tables: B requests of lo .. hi tokens; new = tokens of this step per request (0: the whole prompt)
        # the verify window of a small batch, pages of 64: latency
        dict(name="tables_step", op="tables", B=32, lo=4096, hi=131072, page=64, new=6, short=False),
        # one slot per page, odd lengths, and not enough free pages for the last requests
        dict(name="tables_token_pages", op="tables", B=17, lo=1, hi=40001, page=1, new=0, short=True),
        # 128 requests join after a restart, contexts of 1024 to 131072 tokens
        dict(name="tables_restart", op="tables", B=128, lo=1024, hi=131072, page=64, new=0, short=False),
        # --- norms and rotation
        # the indexer's 64 queries and its key of one draft row, float32 in, FP8 out: latency
        dict(name="rope_indexer_row", op="rope", kind="indexer", T=1, Hq=64, Hk=1, D=128, rot=64, dtype="float32",
             cache="fp8", interleaved=False),
        # the same for a 128 x 6 row verify step
        dict(name="rope_indexer_decode", op="rope", kind="indexer", T=768, Hq=64, Hk=1, D=128, rot=64, dtype="bfloat16",
             cache="fp8", interleaved=False),
        # a prompt chunk of grouped heads, each query and key head normed, from one fused projection into a bf16 cache
        dict(name="rope_heads_prompt", op="rope", kind="heads", T=8192, Hq=32, Hk=8, D=128, rot=128, dtype="bfloat16",
             cache="bfloat16", interleaved=False),
        # odd in every direction: 5 heads of 90 values, 50 of them rotated, float32
        dict(name="rope_heads_odd", op="rope", kind="heads", T=1237, Hq=5, Hk=1, D=90, rot=50, dtype="float32",
             cache="float32", interleaved=True),
        # a prompt chunk's rope queries of 128 heads and its latent rows into the 656-byte FP8 cache
        dict(name="rope_latent_prompt", op="rope", kind="latent", T=16384, Hq=128, Hk=1, D=576, rot=64, dtype="bfloat16",
             cache="fp8_rows", interleaved=True),
        # --- attention over the 4-bit latent cache (128 heads, 2048 selected positions in the models' configurations)
        # one draft row of one long request: latency
        dict(name="mla4_one_row", op="mla4", B=1, W=1, H=128, n=2048, lo=100000, hi=100000, page=0),
        # few heads, a short list, ragged short contexts that leave most of the list empty
        dict(name="mla4_odd", op="mla4", B=11, W=7, H=16, n=500, lo=1, hi=3001, page=16),
        # the verify step of 32 requests, 64-token pages
        dict(name="mla4_verify", op="mla4", B=32, W=6, H=128, n=2048, lo=4096, hi=65536, page=64),
        # the verify step of 128 requests, contiguous cache
        dict(name="mla4_decode", op="mla4", B=128, W=6, H=128, n=2048, lo=1024, hi=131072, page=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "mla4", "mla4"])
    if op == "tables":
        while True:
            lo = _log_int(rng, 1, 8192)
            case = dict(op="tables", B=_log_int(rng, 1, 1024), lo=lo, hi=_log_int(rng, lo, 131072),
                        page=rng.choice([1, 16, 64, 256]), new=rng.choice([0, rng.randint(1, 8)]), short=rng.random() < 0.2)
            if sum(_lengths(case)) <= 3_400_000 and case["B"] * _stride(case) <= 4_000_000:
                return case
    if op == "rope":
        while True:
            kind = rng.choice(["indexer", "heads", "heads", "latent"])
            T, inter = _log_int(rng, 1, 16384), rng.random() < 0.5
            if kind == "indexer":
                case = dict(op="rope", kind=kind, T=T, Hq=rng.choice([32, 64]), Hk=1, D=128, rot=rng.choice([64, 128]),
                            dtype=rng.choice(["bfloat16", "float32"]), cache="fp8", interleaved=inter)
            elif kind == "heads":
                Hk = rng.randint(1, 8)
                D = rng.choice([64, 96, 128, 256, rng.randint(8, 256)])
                dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
                case = dict(op="rope", kind=kind, T=T, Hq=Hk * rng.randint(1, 8), Hk=Hk, D=D,
                            rot=rng.choice([D // 2 * 2, 2 * rng.randint(1, D // 2)]), dtype=dtype, cache=dtype,
                            interleaved=inter)
            else:
                case = dict(op="rope", kind=kind, T=T, Hq=rng.choice([16, 64, 128]), Hk=1, D=576, rot=64, dtype="bfloat16",
                            cache=rng.choice(["bfloat16", "fp8_rows"]), interleaved=inter)
            if work(case)["bytes"] <= work(listed()[7])["bytes"]:
                return case
    while True:
        lo = _log_int(rng, 1, 65536)
        case = dict(op="mla4", B=_log_int(rng, 1, 128), W=rng.randint(1, 6), H=rng.choice([16, 64, 128, 128]),
                    n=_log_int(rng, 64, 2048), lo=lo, hi=_log_int(rng, lo, 131072), page=rng.choice([0, 1, 16, 64]))
        if case["B"] * case["W"] * case["H"] * case["n"] <= 768 * 128 * 2048 and sum(_lengths(case)) <= 3_400_000:
            return case


def _lengths(case):
    """The requests' lengths: evenly spaced over the logarithm of the range, the largest first."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [int(round(hi * (lo / hi) ** (b / max(B - 1, 1)))) for b in range(B)]


def _pages(n, page):
    return -(-n // page)


def _stride(case):
    return _pages(case["hi"] + case["new"], case["page"])


def _new_tokens(case):
    return case["B"] * case["new"] if case["new"] else sum(_lengths(case))


def work(case):
    if case["op"] == "tables":
        B, page, T = case["B"], case["page"], _new_tokens(case)
        L = _lengths(case)
        if case["new"]:      # grown in place
            taken = sum(_pages(n + case["new"], page) - _pages(n, page) for n in L)
            by = 8 * taken
        else:                # built: every entry of the table is written
            by = 4 * sum(_pages(n, page) for n in L) + 4 * B * _stride(case)
        return {"bytes": by + B * (8 + 8 + 4 + (8 if case["new"] else 0)) + 16 * T + 8, "flops": 4 * T}
    if case["op"] == "rope":
        T, Hq, Hk, D, rot = (case[k] for k in ("T", "Hq", "Hk", "D", "rot"))
        size = 2 if case["dtype"] == "bfloat16" else 4
        if case["kind"] == "indexer":
            each = (Hq + Hk) * (D * size + D + 4)
        elif case["kind"] == "heads":
            each = (Hq + Hk) * D * 2 * size
        else:
            each = Hq * rot * 4 + D * 2 + (D * 2 if case["cache"] == "bfloat16" else 656)
        return {"bytes": T * (each + 8 + 8 + 4 * rot), "flops": T * (Hq + Hk) * 8 * (rot if case["kind"] == "latent" else D)}
    R, H, n = case["B"] * case["W"], case["H"], case["n"]
    L = _lengths(case)
    seen = sum(min(n, m + w + 1) for m in L for w in range(case["W"]))
    rows = min(seen, sum(L) + R)
    return {"bytes": rows * ROW4 + R * H * (576 + 512) * 2 + R * n * 4 + R * (576 * 2 + ROW4), "flops": 2 * H * seen * (576 + 512)}


# --------------------------------------------------------------------------- inputs

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt) % (1 << 62))


def _shuffled(g, values):
    perm = torch.randperm(len(values), generator=g, device="cuda")
    return torch.tensor(values, dtype=torch.int64, device="cuda")[perm]


def _offsets(counts):
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return torch.cat([zero, counts.cumsum(0)])


def _prepare_tables(case, seed):
    g = _gen(seed, 1)
    B, page, new, stride = case["B"], case["page"], case["new"], _stride(case)
    length = _shuffled(g, _lengths(case))
    st = dict(case=case, new_len=length + new, old_len=length if new else None)
    held = _pages(length, page) if new else torch.zeros(B, dtype=torch.int64, device="cuda")
    need = _pages(length + new, page) - held
    n_held, n_need = int(held.sum()), int(need.sum())
    ids = torch.randperm(n_held + n_need + 64, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, stride), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(stride, device="cuda") < held[:, None]] = ids[:n_held]
    st["table"] = table
    st["free"] = ids[n_held:].contiguous()
    st["n_free"] = torch.tensor([n_need * 3 // 4 if case["short"] else n_need + 64], dtype=torch.int32, device="cuda")
    counts = torch.full((B,), new, dtype=torch.int64, device="cuda") if new else length
    st["offsets"] = _offsets(counts).to(torch.uint32)
    T = _new_tokens(case)
    st["slots"] = torch.empty(T, dtype=torch.int64, device="cuda")
    st["positions"] = torch.empty(T, dtype=torch.int64, device="cuda")
    st["lengths"] = torch.empty(B, dtype=torch.int64, device="cuda")
    st["n_free_out"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return st


def _rope_table(n_pos, rot, base=10000.0):
    """[n_pos, rot] float32, cosines then sines, the angles in 64 bits."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _prepare_rope(case, seed):
    g = _gen(seed, 2)
    T, Hq, Hk, D, rot, kind = (case[k] for k in ("T", "Hq", "Hk", "D", "rot", "kind"))
    dt = getattr(torch, case["dtype"])
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n_pos = 32768
    st = dict(case=case, cos_sin=_rope_table(n_pos, rot), positions=torch.randint(0, n_pos, (T,), generator=g, device="cuda"))
    pool = 2 * T + 5
    st["slots"] = torch.randperm(pool, generator=g, device="cuda")[:T]
    if kind == "indexer":
        st["q"] = (randn(T, Hq, D) * (0.5 + 2 * torch.rand(Hq, 1, generator=g, device="cuda"))).to(dt)
        st["k"] = (randn(T, Hk, D) * 3 + 0.5).to(dt)
        st["k_weight"] = 1 + 0.2 * randn(D)
        st["k_bias"] = 0.1 * randn(D)
        st["q_out"] = torch.empty(T, Hq, D, dtype=torch.uint8, device="cuda")
        st["q_scale"] = torch.empty(T, Hq, dtype=torch.float32, device="cuda")
        st["k_out"] = torch.zeros(pool, D, dtype=torch.uint8, device="cuda")
        st["k_scale"] = torch.zeros(pool, dtype=torch.float32, device="cuda")
    elif kind == "heads":
        qkv = (randn(T, Hq + 2 * Hk, D) * (0.3 + 3 * torch.rand(D, generator=g, device="cuda"))).to(dt)
        st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        st["q_weight"], st["k_weight"] = 1 + 0.2 * randn(D), 1 + 0.2 * randn(D)
        st["q_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
        st["k_out"] = torch.zeros(pool, Hk, D, dtype=dt, device="cuda")
    else:
        st["q"] = randn(T, Hq, 128 + rot).to(dt)[:, :, 128:]           # the rope part of each query head
        st["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")[:, :, D - rot:]
        kv = randn(T, D) * 2
        kv[:, torch.randint(0, D - rot, (4,), generator=g, device="cuda")] *= 12
        st["k"] = kv.to(dt)
        st["k_weight"] = 0.5 + torch.rand(D - rot, generator=g, device="cuda")
        st["k_out"] = torch.zeros(pool, 656, dtype=torch.uint8, device="cuda") if case["cache"] == "fp8_rows" else \
            torch.zeros(pool, D, dtype=dt, device="cuda")
    return st


def _pack4(x):
    """Latent rows [T, 576] -> rows of 416 bytes: the scale is amax / 6 to the nearest scale value, the code x / scale to the
    nearest magnitude (quotients in float32, ties to the even code)."""
    v = x[:, :512].float().view(-1, 32, 16)
    t = v.abs().amax(2) / 6
    bits = t.view(torch.int32)
    code = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - 8 * (127 - 16)     # rounded to 3 bits of mantissa
    code = torch.where(code > 0, code.clamp(max=254), (t > 4.5 * 2.0 ** -19).int()).to(torch.uint8)
    scale = _scale4(code)
    y = (v / torch.where(scale > 0, scale, torch.ones_like(scale))[:, :, None]).abs()
    m = torch.zeros_like(y)
    for i, edge in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        m += y >= edge if i % 2 else y > edge
    nib = (m + 8 * torch.signbit(v)).to(torch.uint8).view(-1, 64, 8)[:, :, TO_NIBBLES].view(-1, 256, 2)
    rope = x[:, 512:].to(torch.bfloat16).contiguous().view(torch.uint8)
    return torch.cat([nib[:, :, 0] | (nib[:, :, 1] << 4), code, rope], 1)


def _scale4(code):
    """The float32 values of scale codes."""
    c = code.int()
    return torch.where(c > 0, (((c >> 3) + 127 - 16) << 23) + ((c & 7) << 20), torch.zeros_like(c)).view(torch.float32)


def _prepare_mla4(case, seed):
    g = _gen(seed, 3)
    B, W, H, n, page = (case[k] for k in ("B", "W", "H", "n", "page"))
    R = B * W
    length = _shuffled(g, _lengths(case))          # committed tokens; the window's W rows follow
    total = length + W
    outlier = 1 + 4 * (torch.rand(576, generator=g, device="cuda") < 0.02)
    latent = lambda m: torch.randn(m, 576, generator=g, device="cuda").mul_(outlier).to(torch.bfloat16)  # noqa: E731
    st = dict(case=case)
    if page:
        held = _pages(total, page)
        width = _pages(case["hi"] + W, page)
        pool = sum(_pages(m + W, page) for m in _lengths(case)) * page
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(width, device="cuda") < held[:, None]] = \
            torch.randperm(pool // page, generator=g, device="cuda").to(torch.int32)
        st["table"], st["start"] = table, None
    else:
        pool = sum(_lengths(case)) + R
        st["table"], st["start"] = None, _offsets(total)[:-1].contiguous()
    cache = torch.empty(pool, ROW4, dtype=torch.uint8, device="cuda")
    step = 1 << 18
    for t in range(0, pool, step):
        cache[t:t + step] = _pack4(latent(min(step, pool - t)))
    st["cache"] = cache
    pos = (length[:, None] + torch.arange(W, device="cuda")).view(-1)
    st["row_pos"] = pos
    st["row_offsets"] = (torch.arange(B + 1, device="cuda") * W).to(torch.uint32)
    u = torch.rand(R, n, generator=g, device="cuda", dtype=torch.float64)
    j = torch.arange(n, device="cuda", dtype=torch.float64)
    visible = (pos + 1)[:, None]
    spread = torch.floor((j + u) * visible / n).long().clamp(max=visible - 1)
    few = torch.where(j < visible, j, torch.full_like(j, -1)).long()
    st["idx"] = torch.where(visible >= n, spread, few).to(torch.int32)
    st["q"] = (torch.randn(R, H, 576, generator=g, device="cuda") * 2.0).to(torch.bfloat16)
    st["new"] = latent(R)
    req = torch.arange(R, device="cuda") // W
    st["slots"] = _slot_of(st, req, pos)
    st["out"] = torch.empty(R, H, 512, dtype=torch.bfloat16, device="cuda")
    return st


def _slot_of(st, req, pos):
    """Pool slot of positions `pos` of requests `req` (through the block table, or contiguous)."""
    page = st["case"]["page"]
    if not page:
        return st["start"][req] + pos
    return st["table"][req, pos // page].long() * page + pos % page


def prepare(case, seed):
    return {"tables": _prepare_tables, "rope": _prepare_rope, "mla4": _prepare_mla4}[case["op"]](case, seed)


# --------------------------------------------------------------------------- one pass

def _plain_tables(st):
    case, page = st["case"], st["case"]["page"]
    new, old = st["new_len"], st["old_len"]
    first = torch.zeros_like(new) if old is None else _pages(old, page)
    need = (_pages(new, page) - first).clamp(min=0)
    incl = need.cumsum(0)
    n_free = st["n_free"].long()
    served = (need == 0) | (incl <= n_free)
    col = torch.arange(st["table"].shape[1], device="cuda")
    take = (n_free - 1 - (incl - need))[:, None] - (col - first[:, None])
    mine = (col >= first[:, None]) & (col < (first + need)[:, None])
    none = torch.full_like(st["table"], -1)
    page_id = torch.where(served[:, None], st["free"][take.clamp(0, len(st["free"]) - 1)], none)
    table = torch.where(mine, page_id, none if old is None else st["table"])
    off = st["offsets"].long()
    t = torch.arange(st["slots"].numel(), device="cuda")
    req = torch.searchsorted(off, t, right=True) - 1
    pos = new[req] - off[req + 1] + t
    entry = table[req, pos // page].long()
    slots = torch.where(entry >= 0, entry * page + pos % page, torch.full_like(pos, -1))
    lengths = torch.where(served, new, torch.zeros_like(new) if old is None else old)
    return dict(table=table, lengths=lengths, n_free=(n_free - (need * served).sum()).to(torch.int32),
                slots=slots, positions=pos)


def _rotate(x, cos_sin, start, rot, interleaved):
    """x [T, H, D] float; the pairs of dims start .. start + rot - 1 by the angles of each token."""
    c, s = cos_sin[:, None, :rot // 2], cos_sin[:, None, rot // 2:]
    y = x[:, :, start:start + rot]
    a, b = (y[:, :, 0::2], y[:, :, 1::2]) if interleaved else (y[:, :, :rot // 2], y[:, :, rot // 2:])
    ra, rb = a * c - b * s, a * s + b * c
    z = torch.stack([ra, rb], 3).flatten(2) if interleaved else torch.cat([ra, rb], 2)
    return torch.cat([x[:, :, :start], z, x[:, :, start + rot:]], 2)


def _rms(x, weight, eps=1e-6):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight


def _quant8(x):
    """Blocks of 128 values (the last dim) -> E4M3 codes as bytes and their scales."""
    scale = x.abs().amax(-1) / 448
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (x / scale.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _rows8(x):
    """Latent rows [T, 576] float -> rows of 656 bytes."""
    codes, scale = _quant8(x[:, :512].view(-1, 4, 128))
    return torch.cat([codes.view(-1, 512), scale.contiguous().view(torch.uint8), x[:, 512:].to(torch.bfloat16).contiguous()
                      .view(torch.uint8)], 1)


def _rope_outputs(case, q_out, k_out, q_scale=None, k_scale=None):
    """What a rope case returns: what is held in 8 bits as E4M3 values beside its scales (views of the buffers)."""
    if case["kind"] == "indexer":
        return dict(q=q_out.view(torch.float8_e4m3fn), q_scale=q_scale, k=k_out.view(torch.float8_e4m3fn), k_scale=k_scale)
    if case["cache"] == "fp8_rows":
        return dict(q=q_out, codes=k_out[:, :512].view(torch.float8_e4m3fn), scales=k_out[:, 512:528].view(torch.float32),
                    rope=k_out[:, 528:].view(torch.bfloat16))
    return dict(q=q_out, k=k_out)


def _plain_rope(st):
    case = st["case"]
    T, Hk, D, rot, inter, kind = (case[k] for k in ("T", "Hk", "D", "rot", "interleaved", "kind"))
    cs = st["cos_sin"][st["positions"]]
    q, k = st["q"].float(), st["k"].float().view(T, Hk, D)
    if kind == "heads":
        q = _rms(q, st["q_weight"])
        k = _rms(k, st["k_weight"])
    elif kind == "indexer":
        k = k - k.mean(2, keepdim=True)
        k = k * torch.rsqrt(k.square().mean(2, keepdim=True) + 1e-6) * st["k_weight"] + st["k_bias"]
    else:
        k = torch.cat([_rms(k[:, :, :D - rot], st["k_weight"]), k[:, :, D - rot:]], 2)
    q = _rotate(q, cs, 0, rot, inter)
    k = _rotate(k, cs, D - rot if kind == "latent" else 0, rot, inter)
    if kind == "indexer":
        codes, scale = _quant8(q)
        st["q_out"].copy_(codes)
        st["q_scale"].copy_(scale)
        codes, scale = _quant8(k.view(T, D))
        st["k_out"][st["slots"]] = codes
        st["k_scale"][st["slots"]] = scale
    else:
        st["q_out"].copy_(q)
        k = k.view(T, -1)
        k = _rows8(k) if case["cache"] == "fp8_rows" else k.to(st["k_out"].dtype)
        st["k_out"].view(len(st["k_out"]), -1)[st["slots"]] = k
    return _rope_outputs(case, st["q_out"], st["k_out"], st.get("q_scale"), st.get("k_scale"))


def _selected(st):
    """Pool rows [R, n] of the selected positions, and which of them there are."""
    idx = st["idx"].long()
    req = (torch.arange(len(idx), device="cuda") // st["case"]["W"])[:, None]
    return _slot_of(st, req, idx.clamp(min=0)), idx >= 0


def _plain_mla4(st):
    H = st["case"]["H"]
    st["cache"][st["slots"]] = _pack4(st["new"])
    rows, there = _selected(st)
    R, n = rows.shape
    raw = st["cache"][rows.view(-1)]
    value = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), device="cuda")
    nib = torch.stack([raw[:, :256] & 15, raw[:, :256] >> 4], 2).view(-1, 64, 8)[:, :, FROM_NIBBLES].view(-1, 32, 16)
    c = torch.empty(R * n, 576, device="cuda")
    c[:, :512] = (value[nib.int()] * _scale4(raw[:, 256:288])[:, :, None]).view(-1, 512)
    c[:, 512:] = raw[:, 288:].contiguous().view(torch.bfloat16).float()
    del nib, raw
    c = c.view(R, n, 576)
    s = torch.bmm(st["q"].float(), c.transpose(1, 2)) * SOFTMAX_SCALE
    s = torch.where(there[:, None, :], s, torch.full((), -math.inf, device="cuda"))
    p = torch.exp(s - s.amax(2, keepdim=True))
    o = torch.bmm(p, c[:, :, :512]) / p.sum(2, keepdim=True)
    return o.to(torch.bfloat16).view(R, H, 512)


def _own(st):
    import mtp_speculative_decode_gb300 as mtpsd
    case = st["case"]
    if case["op"] == "tables":
        mtpsd.block_table_grow(st["table"], case["page"], st["new_len"], st["free"], st["n_free"], old_len=st["old_len"],
                               lengths=st["lengths"], n_free_out=st["n_free_out"], token_offsets=st["offsets"],
                               slots=st["slots"], positions=st["positions"])
        return dict(table=st["table"], lengths=st["lengths"], n_free=st["n_free_out"], slots=st["slots"],
                    positions=st["positions"])
    if case["op"] == "rope":
        D, rot, kind = case["D"], case["rot"], case["kind"]
        mtpsd.norm_rope(st["positions"], st["cos_sin"], q=st["q"], k=st["k"], interleaved=case["interleaved"], eps=1e-6,
                        q_norm="rms" if kind == "heads" else None, q_weight=st.get("q_weight"),
                        k_norm="layer" if kind == "indexer" else "rms", k_weight=st["k_weight"], k_bias=st.get("k_bias"),
                        k_norm_dim=D - rot if kind == "latent" else None, k_rot_start=D - rot if kind == "latent" else 0,
                        q_out=st["q_out"], q_scale=st.get("q_scale"), k_out=st["k_out"], k_scale=st.get("k_scale"),
                        slots=st["slots"])
        return _rope_outputs(case, st["q_out"], st["k_out"], st.get("q_scale"), st.get("k_scale"))
    mtpsd.pack_latent_fp4(st["new"], st["cache"], slots=st["slots"])
    return mtpsd.sparse_mla_decode(st["q"], st["cache"], st["start"], st["row_offsets"], st["row_pos"], st["idx"], SOFTMAX_SCALE,
                                   out=st["out"], paged=(st["table"], case["page"]) if case["page"] else None)


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "rope": _plain_rope, "mla4": _plain_mla4}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- the definition in 64 bits

def _exact_tables(st):
    """Request by request, handing out the free list from its end."""
    case, page = st["case"], st["case"]["page"]
    B = case["B"]
    free, left = st["free"].tolist(), int(st["n_free"])
    new = st["new_len"].tolist()
    old = [0] * B if st["old_len"] is None else st["old_len"].tolist()
    off = st["offsets"].tolist()
    table = torch.full_like(st["table"], -1) if st["old_len"] is None else st["table"].clone()
    lengths, slots, positions, shut = [], [], [], False
    for b in range(B):
        lo, hi = -(-old[b] // page), -(-new[b] // page)
        shut = shut or hi - lo > left
        ok = hi <= lo or not shut
        if hi > lo:
            ids = free[left - (hi - lo):left][::-1] if ok else [-1] * (hi - lo)
            table[b, lo:hi] = torch.tensor(ids, dtype=torch.int32, device="cuda")
            left -= hi - lo if ok else 0
        lengths.append(new[b] if ok else old[b])
        m = off[b + 1] - off[b]
        pos = torch.arange(new[b] - m, new[b], device="cuda")
        positions.append(pos)
        entry = table[b].long()[pos // page]
        slots.append(torch.where(entry < 0, -1, entry * page + pos % page))
    return dict(table=table, lengths=torch.tensor(lengths, device="cuda"),
                n_free=torch.tensor([left], dtype=torch.int32, device="cuda"), slots=torch.cat(slots),
                positions=torch.cat(positions))


def _turned(x, st, start):
    """x [T, H, D] as complex numbers times the angles'."""
    rot = st["case"]["rot"]
    cs = st["cos_sin"][st["positions"]].double()
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]
    y = x[:, :, start:start + rot]
    if st["case"]["interleaved"]:
        z = torch.view_as_real(torch.view_as_complex(y.contiguous().view(*y.shape[:2], -1, 2)) * turn).flatten(2)
    else:
        w = torch.complex(y[:, :, :rot // 2].contiguous(), y[:, :, rot // 2:].contiguous()) * turn
        z = torch.cat([w.real, w.imag], 2)
    x = x.clone()
    x[:, :, start:start + rot] = z
    return x


def _grid8(y):
    """The nearest E4M3 values of |y| <= 448, ties to even, in 64 bits."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -12))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_rope(st):
    case = st["case"]
    T, Hq, Hk, D, rot, kind = (case[k] for k in ("T", "Hq", "Hk", "D", "rot", "kind"))

    def norm(x, w, b=None, centre=False):
        mean = x.sum(-1, keepdim=True) / x.shape[-1] if centre else 0.0
        var = ((x - mean) ** 2).sum(-1, keepdim=True) / x.shape[-1]
        y = (x - mean) / torch.sqrt(var + 1e-6) * w.double()
        return y if b is None else y + b.double()

    q, k = st["q"].double(), st["k"].double().reshape(T, Hk, D)
    if kind == "heads":
        q, k = norm(q, st["q_weight"]), norm(k, st["k_weight"])
    elif kind == "indexer":
        k = norm(k, st["k_weight"], st["k_bias"], True)
    else:
        k = k.clone()
        k[:, :, :512] = norm(k[:, :, :512], st["k_weight"])
    q, k = _turned(q, st, 0), _turned(k, st, D - rot if kind == "latent" else 0).view(T, -1)
    pool = len(st["k_out"])

    def at_slots(x):
        y = torch.zeros(pool, *x.shape[1:], dtype=torch.float64, device="cuda")
        return y.index_copy_(0, st["slots"], x)

    if kind == "indexer":
        sq, sk = q.abs().amax(2) / 448, k.abs().amax(1) / 448
        return dict(q=_grid8(q / sq[:, :, None]), q_scale=sq, k=at_slots(_grid8(k / sk[:, None])), k_scale=at_slots(sk))
    if case["cache"] == "fp8_rows":
        c = k[:, :512].view(T, 4, 128)
        s = c.abs().amax(2) / 448
        return dict(q=q, codes=at_slots(_grid8(c / s[:, :, None]).view(T, 512)), scales=at_slots(s), rope=at_slots(k[:, 512:]))
    return dict(q=q, k=at_slots(k).view(st["k_out"].shape))


def _unpack4(raw):
    """Rows of 416 bytes [n, 416] -> latent rows [n, 576] in 64 bits, from the bits."""
    b = raw[:, :256].long().view(-1, 64, 4)
    word = b[:, :, 0] + (b[:, :, 1] << 8) + (b[:, :, 2] << 16) + (b[:, :, 3] << 24)
    nib = torch.stack([(word >> (4 * (v // 2) + 16 * (v % 2))) % 16 for v in range(8)], 2).view(len(raw), 512)
    e, m = (nib % 8) // 2, nib % 2
    mag = torch.where(e > 0, (1 + m.double() / 2) * torch.exp2(e.double() - 1), m.double() / 2)
    c = raw[:, 256:288].long()
    scale = torch.where(c > 0, (8 + c % 8).double() * torch.exp2((c // 8).double() - 19), torch.zeros((), device="cuda").double())
    val = torch.where(nib >= 8, -mag, mag) * scale.repeat_interleave(16, 1)
    return torch.cat([val, raw[:, 288:].contiguous().view(torch.bfloat16).double()], 1)


def _nearest4(x):
    """Latent rows [T, 576] as a 4-bit cache holds them, by the distance to every scale and every magnitude."""
    v = x[:, :512].double().view(-1, 32, 16)
    c = torch.arange(1, 255, device="cuda")
    grid = torch.cat([torch.zeros(1, dtype=torch.float64, device="cuda"), (8 + c % 8).double() * torch.exp2((c // 8).double() - 19)])
    # amax / 6 is a float32 quotient by definition
    t = (v.abs().amax(2).float() / 6).double()
    even = lambda n: 1 + (torch.arange(n, device="cuda") % 2).double() * 1e-12  # noqa: E731  (a tie goes to the even code)
    scale = grid[((t[:, :, None] - grid).abs() * even(255)).argmin(2)]
    mags = torch.tensor(MAGNITUDES, dtype=torch.float64, device="cuda")
    y = (v / torch.where(scale > 0, scale, torch.ones_like(scale))[:, :, None]).float().double()   # a float32 quotient too
    far = (y.abs()[..., None] - mags).abs() * even(8)
    near = mags[far.argmin(3)] * torch.where(y < 0, -1.0, 1.0) * scale[:, :, None]
    return torch.cat([near.view(-1, 512), x[:, 512:].to(torch.bfloat16).double()], 1)


def _exact_mla4(st):
    case = st["case"]
    W = case["W"]
    new = _nearest4(st["new"])
    rows, there = _selected(st)
    pos = st["row_pos"]
    out = []
    for r in range(len(rows)):
        keep = rows[r][there[r]]
        at = st["idx"][r].long()[there[r]]
        c = _unpack4(st["cache"][keep])
        b = r // W                                  # the window's rows of this request come from the step itself
        w = at - pos[b * W]
        c = torch.where((w >= 0)[:, None], new[b * W + w.clamp(min=0)], c)
        s = st["q"][r].double() @ c.t() * SOFTMAX_SCALE
        out.append(torch.softmax(s, 1) @ c[:, :512])
    return torch.stack(out)


def exact(case, seed):
    return {"tables": _exact_tables, "rope": _exact_rope, "mla4": _exact_mla4}[case["op"]](prepare(case, seed))
