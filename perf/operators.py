"""The operators that lead from the verify rows' hidden states to the acceptance of the drafts, as cases to measure.

Three operators, in the order in which a decode step runs them:

``gemm``    matrix product of FP8 E4M3 codes with a float32 scale for each block of 128 (a projection, or the language
            model's head): out[m, n] = sum_kb sa[m, kb] * sw[n, kb] * sum_{k in block kb} a[m, k] * w[n, k].
``logits``  penalties for repeated tokens, biases and the grammar mask on the logits of every verify row, then the greedy
            token and the target distribution that the acceptance reads.
``counts``  the token table that the penalties read: built from the requests' histories when they join, and advanced by
            the accepted tokens of a step.

``run`` computes a case in plain torch operations, or with the framework's kernels where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

SEEN = -32768          # the table word's sign bit: the token occurs in the prompt; the low 15 bits count outputs
COUNT_MAX = 32767


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # --- projections and the head (sizes: hidden 6144, the 12288 -> 6144 draft-input projection, vocabulary 154880)
        # one draft row through the 6144 -> 576 latent projection: the smallest call, latency and weight reads
        dict(name="gemm_latent_one_row", op="gemm", M=1, N=576, K=6144, w_rows=1, out="float32"),
        # the draft input projection for the 64 requests of a draft step: weight reads
        dict(name="gemm_draft_input", op="gemm", M=64, N=6144, K=12288, w_rows=128, out="bfloat16"),
        # ragged in every direction: 77 rows, 2049 outputs, the quantizer's own 1 x 128 weight blocks
        dict(name="gemm_ragged", op="gemm", M=77, N=2049, K=1920, w_rows=1, out="float32"),
        # head of a 32 x 6 row verify step: a 951 MB weight read
        dict(name="gemm_head_verify", op="gemm", M=192, N=154880, K=6144, w_rows=128, out="bfloat16"),
        # head of a 128 x 6 row verify step: compute bound
        dict(name="gemm_head_decode", op="gemm", M=768, N=154880, K=6144, w_rows=128, out="bfloat16"),
        # --- logits to the acceptance's inputs
        # one request without drafts, a small vocabulary, penalties and temperature: latency
        dict(name="logits_one_row", op="logits", B=1, K=0, V=32000, logits="bfloat16", penalties=True, bias=0, mask="none",
             probs=True, processed=False),
        # odd vocabulary, everything on, the processed logits kept too
        dict(name="logits_odd_all", op="logits", B=17, K=3, V=50001, logits="float32", penalties=True, bias=300, mask="all",
             probs=True, processed=True),
        # the verify step's rejection sampling: float32 logits, penalties, a third of the requests under a grammar
        dict(name="logits_verify", op="logits", B=32, K=5, V=154880, logits="float32", penalties=True, bias=40, mask="some",
             probs=True, processed=False),
        # the greedy decode step of 128 requests: only the argmax leaves the kernel
        dict(name="logits_greedy", op="logits", B=128, K=5, V=154880, logits="bfloat16", penalties=True, bias=0, mask="some",
             probs=False, processed=False),
        # --- the token table
        # two short requests join
        dict(name="counts_short", op="counts", B=2, lo=100, hi=300, V=1000, K=3),
        # a batch of 128 joins after a restart, contexts of 1024 to 131072 tokens, then commits a step
        dict(name="counts_decode", op="counts", B=128, lo=1024, hi=131072, V=154880, K=5),
        # few very long contexts
        dict(name="counts_long", op="counts", B=8, lo=4096, hi=1048576, V=154880, K=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "logits", "logits", "counts"])
    if op == "gemm":
        while True:
            M, N, K = _log_int(rng, 1, 1024), _log_int(rng, 64, 154880), 128 * _log_int(rng, 1, 96)
            if M * N * K <= 768 * 154880 * 6144:
                return dict(op="gemm", M=M, N=N, K=K, w_rows=rng.choice([1, 128]), out=rng.choice(["bfloat16", "float32"]))
    if op == "logits":
        while True:
            B, K, V = _log_int(rng, 1, 128), rng.randint(0, 7), _log_int(rng, 1000, 200000)
            if B * (K + 1) * V <= 768 * 154880:
                return dict(op="logits", B=B, K=K, V=V, logits=rng.choice(["bfloat16", "float32"]),
                            penalties=rng.random() < 0.75, bias=rng.choice([0, rng.randint(1, 300)]),
                            mask=rng.choice(["none", "some", "all"]), probs=rng.random() < 0.7, processed=rng.random() < 0.2)
    lo = _log_int(rng, 1, 8192)
    return dict(op="counts", B=_log_int(rng, 1, 128), lo=lo, hi=_log_int(rng, lo, 131072), V=_log_int(rng, 1000, 200000),
                K=rng.randint(0, 7))


def _lengths(case):
    """Context lengths of a counts case: evenly spaced over the logarithm of the range, the largest first."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [int(round(hi * (lo / hi) ** (b / max(B - 1, 1)))) for b in range(B)]


def _ld(V):
    return (V + 7) // 8 * 8


def _mask_rows(case):
    """Which rows of a logits case have a mask: none, those of every third request, or all."""
    B, W = case["B"], case["K"] + 1
    use = {"none": lambda b: False, "some": lambda b: b % 3 == 0, "all": lambda b: True}[case["mask"]]
    rows, n = [], 0
    for b in range(B):
        for _ in range(W):
            rows.append(n if use(b) else -1)
            n += use(b)
    return rows, n


def work(case):
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = K // 128
        sw = N if case["w_rows"] == 1 else -(-N // 128)
        return {"bytes": M * K + 4 * M * kb + N * K + 4 * sw * kb + M * N * (2 if case["out"] == "bfloat16" else 4),
                "flops": 2 * M * N * K}
    if case["op"] == "logits":
        R, V = case["B"] * (case["K"] + 1), case["V"]
        by = R * V * (2 if case["logits"] == "bfloat16" else 4) + R * 8
        by += case["B"] * V * 2 if case["penalties"] else 0
        by += case["B"] * case["bias"] * 8 + _mask_rows(case)[1] * (V // 8)
        by += R * V * 4 * (case["probs"] + case["processed"])
        return {"bytes": by, "flops": R * V * (5 if case["probs"] else 2)}
    S = sum(_lengths(case))
    return {"bytes": 8 * S + 2 * case["B"] * _ld(case["V"]), "flops": S}


# --------------------------------------------------------------------------- inputs

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt) % (1 << 62))


def _quantize(x):
    """float32 [rows, K] -> E4M3 codes (uint8) and the scales of its 1 x 128 blocks."""
    rows, K = x.shape
    xb = x.view(rows, K // 128, 128)
    scale = xb.abs().amax(2) / 448
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = (xb / scale.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(rows, K), scale


def _quantize_weight(g, N, K, w_rows):
    codes = torch.empty(N, K, dtype=torch.uint8, device="cuda")
    n_sc = N if w_rows == 1 else -(-N // 128)
    scales = torch.empty(n_sc, K // 128, dtype=torch.float32, device="cuda")
    step = 16384
    for n0 in range(0, N, step):
        n1 = min(N, n0 + step)
        x = torch.randn(n1 - n0, K, generator=g, device="cuda") * (1.0 / math.sqrt(K))
        if w_rows == 1:
            codes[n0:n1], scales[n0:n1] = _quantize(x)
            continue
        rows = -(-(n1 - n0) // 128)
        pad = torch.zeros(rows * 128, K, device="cuda")
        pad[:n1 - n0] = x
        xb = pad.view(rows, 128, K // 128, 128)
        s = xb.abs().amax((1, 3)) / 448
        q = (xb / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(rows * 128, K)
        codes[n0:n1] = q[:n1 - n0]
        scales[n0 // 128:n0 // 128 + rows] = s
    return codes, scales


def _zipf_tokens(g, n, V):
    """Token ids with the skew of text: id = V^u - 1 under a random relabelling of the vocabulary."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(V)) - 1).long().clamp(0, V - 1)
    return (ids * 7919 + 13) % V


def _prepare_gemm(case, seed):
    g = _gen(seed, 1)
    M, N, K = case["M"], case["N"], case["K"]
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, torch.randint(0, K, (max(1, K // 512),), generator=g, device="cuda")] *= 20   # outlier channels of a hidden state
    a, sa = _quantize(x)
    w, sw = _quantize_weight(g, N, K, case["w_rows"])
    return dict(case=case, a=a, sa=sa, w=w, sw=sw, out=torch.empty(M, N, dtype=getattr(torch, case["out"]), device="cuda"))


def _prepare_logits(case, seed):
    g = _gen(seed, 2)
    B, K, V = case["B"], case["K"], case["V"]
    W, R = K + 1, case["B"] * (case["K"] + 1)
    st = dict(case=case)
    x = torch.randn(R, V, generator=g, device="cuda") * 2.5
    peaks = torch.randint(0, V, (R, 8), generator=g, device="cuda")
    x.scatter_add_(1, peaks, torch.rand(R, 8, generator=g, device="cuda") * 14)
    st["logits"] = x.to(getattr(torch, case["logits"]))
    st["row_offsets"] = (torch.arange(B + 1, dtype=torch.int64) * W).to(torch.uint32).cuda()
    st["draft"] = _zipf_tokens(g, B * K, V).view(B, K)
    st["temperature"] = torch.rand(B, generator=g, device="cuda") * 0.9 + 0.4
    st["temperature"][::4] = 0.0 if B > 1 else 0.7     # every fourth request decodes greedily
    if case["penalties"]:
        n = 2048
        tok = _zipf_tokens(g, B * n, V).view(B, n)
        cnt = torch.zeros(B, _ld(V), dtype=torch.int32, device="cuda")
        cnt.scatter_add_(1, tok[:, n // 2:], torch.ones(B, n - n // 2, dtype=torch.int32, device="cuda"))
        seen = torch.zeros(B, _ld(V), dtype=torch.bool, device="cuda")
        seen.scatter_(1, tok[:, :n // 2], True)
        st["counts"] = (cnt.clamp(max=COUNT_MAX) + torch.where(seen, SEEN, 0)).to(torch.int16)
        st["repetition"] = 1.0 + torch.rand(B, generator=g, device="cuda") * 0.3
        st["frequency"] = torch.rand(B, generator=g, device="cuda") * 0.5
        st["presence"] = torch.rand(B, generator=g, device="cuda") * 0.8
    if case["bias"]:
        n = case["bias"]
        ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:n] for _ in range(B)])
        n = ids.shape[1]
        st["bias_offsets"] = (torch.arange(B + 1, dtype=torch.int64) * n).to(torch.uint32).cuda()
        st["bias_tokens"] = ids.reshape(-1).to(torch.int32).contiguous()
        st["bias_values"] = torch.rand(B * n, generator=g, device="cuda") * 12 - 6
    if case["mask"] != "none":
        rows, n = _mask_rows(case)
        words = -(-V // 32)
        st["mask_rows"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
        bits = torch.randint(-2 ** 31, 2 ** 31, (n, words), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        few = torch.arange(n, device="cuda") % 2 == 0       # half the grammar states allow a handful of tokens
        keep = torch.zeros(n, words * 32, dtype=torch.bool, device="cuda")
        keep.scatter_(1, torch.randint(0, V, (n, 24), generator=g, device="cuda"), True)
        sh = torch.arange(32, device="cuda", dtype=torch.int64)
        narrow = (keep.view(n, words, 32).long() << sh).sum(2)
        narrow = torch.where(narrow >= 2 ** 31, narrow - 2 ** 32, narrow).to(torch.int32)
        st["bitmask"] = torch.where(few[:, None], narrow, bits).contiguous()
    st["argmax"] = torch.empty(R, dtype=torch.int64, device="cuda")
    st["probs"] = torch.empty(R, V, dtype=torch.float32, device="cuda") if case["probs"] else None
    st["processed"] = torch.empty(R, V, dtype=torch.float32, device="cuda") if case["processed"] else None
    return st


def _prepare_counts(case, seed):
    g = _gen(seed, 3)
    B, V, K = case["B"], case["V"], case["K"]
    L = _lengths(case)
    st = dict(case=case, lengths=L)
    st["tokens"] = _zipf_tokens(g, sum(L), V)
    st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(L)]).astype(np.uint32)).cuda()
    st["n_prompt"] = torch.tensor([(3 * n) // 4 for n in L], dtype=torch.int64, device="cuda")
    st["draft"] = _zipf_tokens(g, B * K, V).view(B, K)
    st["num_accepted"] = torch.randint(0, K + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    st["next_tokens"] = _zipf_tokens(g, B, V)
    st["table"] = torch.zeros(B, _ld(V), dtype=torch.int16, device="cuda")
    return st


def prepare(case, seed):
    return {"gemm": _prepare_gemm, "logits": _prepare_logits, "counts": _prepare_counts}[case["op"]](case, seed)


# --------------------------------------------------------------------------- one pass

def _plain_gemm(st):
    N, K = st["w"].shape
    a = st["a"].view(torch.float8_e4m3fn).float() * st["sa"].repeat_interleave(128, 1)
    sw = st["sw"] if st["sw"].shape[0] == N else st["sw"].repeat_interleave(128, 0)[:N]
    w = st["w"].view(torch.float8_e4m3fn).float()
    w.view(N, K // 128, 128).mul_(sw.unsqueeze(2))
    return (a @ w.t()).to(st["out"].dtype)


def _allowed(st, R, V):
    """[R, V] truth values of the grammar masks."""
    rows = st["mask_rows"].long()
    sh = torch.arange(32, device="cuda", dtype=torch.int32)
    bits = (st["bitmask"].unsqueeze(2) >> sh).bitwise_and(1).bool().view(st["bitmask"].shape[0], -1)[:, :V]
    return torch.where((rows >= 0)[:, None], bits[rows.clamp(min=0)], torch.ones((), dtype=torch.bool, device="cuda"))


def _plain_logits(st):
    case = st["case"]
    B, K, V = case["B"], case["K"], case["V"]
    W, R = K + 1, B * (K + 1)
    req = torch.arange(R, device="cuda") // W
    x = st["logits"].float()
    if case["penalties"]:
        word = st["counts"][:, :V].int()
        count = (word & COUNT_MAX)[req]
        seen = (word < 0)[req]
        for j in range(K):      # row i of a request follows its first i drafts
            rows = torch.nonzero(torch.arange(R, device="cuda") % W > j).flatten()
            count[rows, st["draft"][req[rows], j]] += 1
        col = lambda t: t[req].unsqueeze(1)  # noqa: E731
        x = torch.where(seen | (count > 0), torch.where(x > 0, x / col(st["repetition"]), x * col(st["repetition"])), x)
        x = x - col(st["frequency"]) * count
        x = x - torch.where(count > 0, col(st["presence"]), torch.zeros((), device="cuda"))
        del count, seen
    if case["bias"]:
        dense = torch.zeros(B, V, device="cuda")
        n = st["bias_tokens"].numel() // B
        dense.scatter_add_(1, st["bias_tokens"].view(B, n).long(), st["bias_values"].view(B, n))
        x = x + dense[req]
    if case["mask"] != "none":
        x = torch.where(_allowed(st, R, V), x, torch.full((), -math.inf, device="cuda"))
    best = x.amax(1, keepdim=True)
    out = dict(argmax=torch.where(x == best, torch.arange(V, device="cuda"), V).amin(1))
    if case["probs"]:
        t = st["temperature"][req].unsqueeze(1)
        e = torch.exp((x - best) / torch.where(t > 0, t, torch.ones_like(t)))
        p = e / e.sum(1, keepdim=True)
        out["probs"] = torch.where(t > 0, p, (torch.arange(V, device="cuda") == out["argmax"][:, None]).float())
    if case["processed"]:
        out["processed"] = x
    return out


def _plain_counts(st):
    case, V, K = st["case"], st["case"]["V"], st["case"]["K"]
    B, L = case["B"], st["lengths"]
    tok = st["tokens"]
    req = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(L, device="cuda"), output_size=len(tok))
    first = st["offsets"].long()[:-1]
    prompt = torch.arange(len(tok), device="cuda") - first[req] < st["n_prompt"][req]
    cell = req * V + tok
    seen = torch.zeros(B * V, dtype=torch.int32, device="cuda").index_add_(0, cell, prompt.int())
    count = torch.zeros(B * V, dtype=torch.int32, device="cuda").index_add_(0, cell, (~prompt).int())
    base = torch.arange(B, device="cuda") * V
    for j in range(K):
        count.index_add_(0, base + st["draft"][:, j], (st["num_accepted"] > j).int())
    count.index_add_(0, base + st["next_tokens"], torch.ones(B, dtype=torch.int32, device="cuda"))
    word = count.clamp(max=COUNT_MAX) + torch.where(seen > 0, SEEN, 0)
    table = torch.zeros_like(st["table"])
    table[:, :V] = word.view(B, V).to(torch.int16)
    return table


def _own(st):
    import mtp_speculative_decode_gb300 as mtpsd
    case = st["case"]
    if case["op"] == "gemm":
        return mtpsd.gemm_fp8_block128(st["a"], st["sa"], st["w"], st["sw"], out=st["out"])
    if case["op"] == "logits":
        mtpsd.process_logits(
            st["logits"], st["row_offsets"], draft=st["draft"] if case["penalties"] else None, counts=st.get("counts"),
            repetition=st.get("repetition"), frequency=st.get("frequency"), presence=st.get("presence"),
            bias_offsets=st.get("bias_offsets"), bias_tokens=st.get("bias_tokens"), bias_values=st.get("bias_values"),
            bitmask=st.get("bitmask"), mask_rows=st.get("mask_rows"), temperature=st["temperature"],
            argmax=st["argmax"], probs=st["probs"], out_logits=st["processed"])
        out = dict(argmax=st["argmax"])
        if case["probs"]:
            out["probs"] = st["probs"]
        if case["processed"]:
            out["processed"] = st["processed"]
        return out
    mtpsd.token_counts_build(st["tokens"], st["offsets"], case["V"], n_prompt=st["n_prompt"], counts=st["table"])
    mtpsd.token_counts_accept(st["table"], case["V"], st["draft"], st["num_accepted"], st["next_tokens"])
    return st["table"]


def run(state):
    if own:
        return _own(state)
    return {"gemm": _plain_gemm, "logits": _plain_logits, "counts": _plain_counts}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- the definition in 64 bits

def _exact_gemm(st):
    M, K = st["a"].shape
    N = st["w"].shape[0]
    code = torch.arange(256, device="cuda")
    e, m = (code >> 3) & 15, code & 7
    val = torch.where(e > 0, (1 + m.double() / 8) * torch.pow(2.0, e.double() - 7), m.double() / 8 * 2.0 ** -6)
    val = torch.where(code >= 128, -val, val)
    out = torch.empty(M, N, dtype=torch.float64, device="cuda")
    a = (val[st["a"].int()].view(M, K // 128, 128) * st["sa"].double()[:, :, None]).view(M, K)
    step = 8192     # a multiple of 128, so that a slice starts at a weight block
    for n0 in range(0, N, step):
        n1 = min(N, n0 + step)
        s = st["sw"][n0:n1] if st["sw"].shape[0] == N else \
            st["sw"][n0 // 128:-(-n1 // 128)].repeat_interleave(128, 0)[:n1 - n0]
        w = (val[st["w"][n0:n1].int()].view(n1 - n0, K // 128, 128) * s.double()[:, :, None]).view(n1 - n0, K)
        out[:, n0:n1] = a @ w.t()
    return out


def _exact_logits(st):
    """Row by row, from the sparse lists instead of dense tables."""
    case = st["case"]
    B, K, V = case["B"], case["K"], case["V"]
    R = B * (K + 1)
    tops = []
    probs = torch.zeros(R, V, dtype=torch.float64, device="cuda") if case["probs"] else None
    processed = torch.empty(R, V, dtype=torch.float64, device="cuda") if case["processed"] else None
    temp = st["temperature"].double().tolist()
    for b in range(B):
        if case["penalties"]:
            word = st["counts"][b, :V].long()
            theta, alpha, beta = (float(st[k][b]) for k in ("repetition", "frequency", "presence"))
        for i in range(K + 1):
            r = b * (K + 1) + i
            x = st["logits"][r].double()
            if case["penalties"]:
                n = word % 32768
                if i:
                    n = n + torch.bincount(st["draft"][b, :i], minlength=V)
                hit = torch.nonzero((word < 0) | (n > 0)).flatten()
                y, n = x[hit], n[hit].double()
                y = torch.where(y > 0, y / theta, y * theta) - alpha * n - beta * (n > 0)
                x = x.index_copy(0, hit, y)
            if case["bias"]:
                n = st["bias_tokens"].numel() // B
                x = x.index_add(0, st["bias_tokens"][b * n:(b + 1) * n].long(),
                                st["bias_values"][b * n:(b + 1) * n].double())
            if case["mask"] != "none":
                m = int(st["mask_rows"][r])
                if m >= 0:
                    t = torch.arange(V, device="cuda")
                    x = x.masked_fill((st["bitmask"][m].long()[t // 32] >> (t % 32)) % 2 == 0, -math.inf)
            best = x.max()
            tops.append(torch.nonzero(x == best)[0, 0])
            if case["probs"]:
                if temp[b] > 0:
                    probs[r] = torch.softmax((x - best) / temp[b], 0)
                else:
                    probs[r, tops[-1]] = 1.0
            if case["processed"]:
                processed[r] = x
    out = dict(argmax=torch.stack(tops))
    if case["probs"]:
        out["probs"] = probs
    if case["processed"]:
        out["processed"] = processed
    return out


def _exact_counts(st):
    """Request by request, by sorting its tokens."""
    case = st["case"]
    table = torch.zeros_like(st["table"])
    o = 0
    for b, n in enumerate(st["lengths"]):
        tok, cut = st["tokens"][o:o + n], int(st["n_prompt"][b])
        done = torch.cat([tok[cut:], st["draft"][b, :int(st["num_accepted"][b])], st["next_tokens"][b:b + 1]])
        ids, cnt = torch.unique(done, return_counts=True)
        row = torch.zeros(table.shape[1], dtype=torch.int64, device="cuda")
        row[ids] = cnt.clamp(max=COUNT_MAX)
        seen = torch.unique(tok[:cut])
        row[seen] = row[seen] + SEEN
        table[b] = row.to(torch.int16)
        o += n
    return table


def exact(case, seed):
    return {"gemm": _exact_gemm, "logits": _exact_logits, "counts": _exact_counts}[case["op"]](prepare(case, seed))
