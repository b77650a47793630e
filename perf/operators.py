"""Cases and plain forms of three operators: whole-prompt attention, the 4-bit K/V store, attention over the 4-bit cache.

Notation: a token's K (or V) of one kv head is a row of d = 128 numbers; query head h reads kv head h // (H_q / H_kv).

prompt      out = softmax(q k^T / sqrt(d)) v over packed sequences of different lengths: the n rows of a sequence that
            holds L tokens are its newest ones, and row i sees its first L - n + i + 1 tokens (n = L: a whole prompt).
store       K/V rows into the 4-bit cache. A group of 16 numbers x has the scale s = E4M3(max|x| / (6 S)) and the
            codes E2M1(x / (s S)), both rounded to nearest, ties to even; S is the layer's scale, a power of two.
attend_fp4  softmax attention of every query row over the tokens of its index set, K and V held in those 4 bits.
"""
import math
from statistics import NormalDist

import torch

own = False  # set by the caller: False runs the plain forms below, True the framework's calls

D = 128
GROUP = 16  # numbers that share a scale


def listed():
    return [
        # one new token for each of 16 conversations whose whole context still fits the sparse budget of 3136 tokens
        dict(name="prompt_one_token", op="prompt", heads=32, kv_heads=4, seqs=16, rows=1, cache=3135, ragged=True,
             fused=False, lse=True),
        # a serving batch of short prompts of different lengths, Q, K and V as views of one fused projection
        dict(name="prompt_ragged", op="prompt", heads=32, kv_heads=4, seqs=24, rows=1500, cache=0, ragged=True, fused=True,
             lse=False),
        # a chunk of 2048 new tokens on a cache of 65536, with the softmax denominators for merging with other parts
        dict(name="prompt_chunk", op="prompt", heads=32, kv_heads=4, seqs=1, rows=2048, cache=65536, ragged=False,
             fused=False, lse=True),
        # one long prompt
        dict(name="prompt_long", op="prompt", heads=32, kv_heads=4, seqs=1, rows=16384, cache=0, ragged=False, fused=False,
             lse=False),
        # a decode step's new tokens: one for each of 16 sequences
        dict(name="store_decode", op="store", kv_heads=4, seqs=16, rows=1, cache=4095, layers=1, ragged=False),
        # draft tokens: four for each of 64 sequences, two layers
        dict(name="store_drafts", op="store", kv_heads=4, seqs=64, rows=4, cache=1020, layers=2, ragged=False),
        # the serving batch of short prompts
        dict(name="store_ragged", op="store", kv_heads=4, seqs=24, rows=1500, cache=0, layers=1, ragged=True),
        # a long prompt's rows
        dict(name="store_long", op="store", kv_heads=4, seqs=1, rows=65536, cache=0, layers=1, ragged=False),
        # one decode row on a short context, one kv head
        dict(name="attend_fp4_tiny", op="attend_fp4", heads=8, kv_heads=1, seqs=1, drafts=1, ctx=4096, layers=1, sink=4,
             window=128, topk=256, hi_block=0, hi_topblocks=0, ragged=False),
        # batched decode at 128K tokens of context
        dict(name="attend_fp4_128k", op="attend_fp4", heads=32, kv_heads=4, seqs=16, drafts=1, ctx=131072, layers=1, sink=64,
             window=1024, topk=2048, hi_block=64, hi_topblocks=256, ragged=False),
        # one decode row at 1M tokens, four layers on one index set
        dict(name="attend_fp4_1m", op="attend_fp4", heads=32, kv_heads=4, seqs=1, drafts=1, ctx=1048576, layers=4, sink=64,
             window=2048, topk=2048, hi_block=128, hi_topblocks=512, ragged=False),
        # ragged serving decode, two layers on one index set
        dict(name="attend_fp4_ragged", op="attend_fp4", heads=32, kv_heads=4, seqs=64, drafts=1, ctx=32768, layers=2, sink=64,
             window=1024, topk=2048, hi_block=64, hi_topblocks=256, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "store", "attend_fp4"])
    if op == "prompt":
        kv = rng.choice([1, 2, 4, 8])
        ratio = rng.choice([1, 2, 4, 8, 16] if kv < 4 else [1, 2, 4, 8])
        seqs = _log(rng, 1, 64)
        # the scores of the plain form, seqs * heads * rows * length, stay within those of the longest listed prompt
        most = 16384 * 16384 * 32 // (kv * ratio * seqs)
        rows = _log(rng, 1, min(8192, int(math.isqrt(most))))
        cache = rng.choice([0, _log(rng, 1, max(1, min(65536, most // rows - rows)))])
        cache = min(cache, 1_000_000 // seqs)
        return dict(op=op, heads=kv * ratio, kv_heads=kv, seqs=seqs, rows=rows, cache=cache, ragged=rng.random() < 0.7,
                    fused=cache == 0 and rng.random() < 0.5, lse=rng.random() < 0.5)
    if op == "store":
        kv, layers = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4])
        seqs = _log(rng, 1, 64)
        rows = _log(rng, 1, 65536 * 4 // (kv * layers * seqs))
        return dict(op=op, kv_heads=kv, seqs=seqs, rows=rows, cache=_log(rng, 1, 65536 // seqs), layers=layers,
                    ragged=rng.random() < 0.7)
    kv = rng.choice([1, 2, 4, 8])
    ratio = rng.choice([1, 2, 4, 8])
    seqs, layers, drafts = _log(rng, 1, 32), rng.choice([1, 2, 4]), rng.choice([1, 1, 1, 4])
    if kv == 8:
        seqs = min(seqs, 8)
    if seqs * drafts > 32:
        drafts = 1
    ctx = _log(rng, 1, 2097152 // (seqs * layers))
    hi = rng.random() < 0.5
    return dict(op=op, heads=kv * ratio, kv_heads=kv, seqs=seqs, drafts=drafts, ctx=ctx, layers=layers, sink=_log(rng, 1, 64),
                window=_log(rng, 16, 2048), topk=_log(rng, 1, 2048), hi_block=64 if hi else 0, hi_topblocks=256 if hi else 0,
                ragged=rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------------------------------------------------------


def _lengths(case):
    """Rows and cached tokens of each sequence, from the case alone. Ragged ones spread over the range: the longest has the
    case's sizes, the shortest one row (or one token)."""
    n, rows, cache = case["seqs"], case["rows"], case["cache"]
    if not case["ragged"] or n == 1:
        return [rows] * n, [cache] * n
    part = [((7 * i) % n + 1) / n for i in range(n)]  # 1/n .. 1, not in order
    return [max(1, round(rows * p * p)) for p in part], [round(cache * p) for p in part]


def _contexts(case):
    """Tokens of each sequence of decode rows: the case's, or lognormal around it as serving traffic is."""
    n = case["seqs"]
    if not case["ragged"] or n == 1:
        return [max(case["ctx"], case["drafts"])] * n
    z = NormalDist()
    lens = [round(case["ctx"] * math.exp(z.inv_cdf(((7 * i) % n + 0.5) / n))) for i in range(n)]
    return [max(case["drafts"], min(1048576, length)) for length in lens]


def _tables(rows, lens, device):
    """First row of each sequence (and the end), first cache row, tokens in the cache."""
    ro, ko = [0], [0]
    for n, length in zip(rows, lens):
        ro.append(ro[-1] + n)
        ko.append(ko[-1] + length)
    return (torch.tensor(ro, dtype=torch.int32, device=device), torch.tensor(ko[:-1], dtype=torch.int64, device=device),
            torch.tensor(lens, dtype=torch.int32, device=device), ro[-1], ko[-1])


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rows(tokens, heads, layers, g):
    """K or V rows as a projection gives them: normal, with a head's channels of different size."""
    size = torch.exp2(torch.randn((heads, D), generator=g, device="cuda") * 0.7)
    return [_normal((tokens, heads, D), g, torch.float32).mul_(size).to(torch.bfloat16) for _ in range(layers)]


def _sets(case, lens, g):
    """Index sets of decode rows: sink, random tokens of the middle (inside random kept blocks with a block pass), window;
    ascending, -1 behind the last."""
    s0, w, k, hb, nb = (case[x] for x in ("sink", "window", "topk", "hi_block", "hi_topblocks"))
    out = []
    for length in lens:
        s = min(s0, length)
        ws = max(s, length - w)
        mid = torch.arange(s, ws, device="cuda")
        if hb and len(mid) > 0:
            first, last = s // hb, (ws - 1) // hb
            keep = torch.rand(last - first + 1, generator=g, device="cuda").topk(min(nb, last - first + 1)).indices + first
            mid = (keep.sort().values[:, None] * hb + torch.arange(hb, device="cuda")).flatten()
            mid = mid[(mid >= s) & (mid < ws)]
        if len(mid) > k:
            mid = mid[torch.rand(len(mid), generator=g, device="cuda").topk(k).indices].sort().values
        whole = torch.cat([torch.arange(s, device="cuda"), mid, torch.arange(ws, length, device="cuda")])
        out.append(torch.nn.functional.pad(whole, (0, s0 + w + k - len(whole)), value=-1))
    return torch.stack(out).to(torch.int32)


def _fp4_cache(tokens, heads, g):
    """Codes and group scales of `tokens` rows: rows drawn from a pool of quantised normal ones."""
    pool = _rows(8192, heads, 1, g)[0]
    codes, scales, _ = _plain_quantise(pool, 2.0 ** -6)
    pick = torch.randint(0, 8192, (tokens,), generator=g, device="cuda")
    return codes[pick], scales[pick]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "prompt":
        H, K = case["heads"], case["kv_heads"]
        rows, cache = _lengths(case)
        lens = [n + c for n, c in zip(rows, cache)]
        st["row_offset"], st["kv_offset"], st["seq_lens"], n_rows, tokens = _tables(rows, lens, "cuda")
        st["max_rows"], st["max_len"], st["n_rows"], st["tokens"] = max(rows), max(lens), n_rows, tokens
        if case["fused"]:  # one projection's output: Q, K and V of a token side by side
            qkv = _normal((n_rows, H + 2 * K, D), g)
            qkv[:, H:H + K] = _rows(n_rows, K, 1, g)[0]
            st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        else:
            st["q"], st["k"], st["v"] = _normal((n_rows, H, D), g), _rows(tokens, K, 1, g)[0], _normal((tokens, K, D), g)
        st["out"] = torch.empty((n_rows, H, D), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((n_rows, H), dtype=torch.float32, device="cuda") if case["lse"] else None
    elif case["op"] == "store":
        K, G = case["kv_heads"], case["layers"]
        rows, cache = _lengths(case)
        lens = [n + c for n, c in zip(rows, cache)]
        st["row_offset"], st["kv_offset"], st["seq_lens"], n_rows, tokens = _tables(rows, lens, "cuda")
        st["max_len"], st["n_rows"], st["tokens"] = max(lens), n_rows, tokens
        st["k_new"], st["v_new"] = _rows(n_rows, K, G, g), _rows(n_rows, K, G, g)
        st["k_scale"], st["v_scale"] = [2.0 ** -6] * G, [2.0 ** -7] * G
        byte = lambda *shape: [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(G)]
        st["k"], st["v"] = byte(tokens, K, D // 2), byte(tokens, K, D // 2)
        st["k_group"], st["v_group"] = byte(tokens, K, D // GROUP), byte(tokens, K, D // GROUP)
        st["k_round"], st["v_round"] = ([torch.empty_like(x) for x in st[n]] for n in ("k_new", "v_new"))
    else:
        H, K, G, drafts = case["heads"], case["kv_heads"], case["layers"], case["drafts"]
        n = case["seqs"]
        lens = _contexts(case)
        _, st["kv_offset"], st["seq_lens"], _, tokens = _tables(lens, lens, "cuda")
        st["tokens"], st["max_len"] = tokens, max(lens)
        q_len = [length - drafts + 1 + j for length in lens for j in range(drafts)]
        st["q_seq"] = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(drafts)
        st["q_len"] = torch.tensor(q_len, dtype=torch.int32, device="cuda")
        st["sets"] = _sets(case, q_len, g)
        st["q"] = [_normal((n * drafts, H, D), g) for _ in range(G)]
        st["k"], st["k_group"] = map(list, zip(*[_fp4_cache(tokens, K, g) for _ in range(G)]))
        st["v"], st["v_group"] = map(list, zip(*[_fp4_cache(tokens, K, g) for _ in range(G)]))
        st["k_scale"], st["v_scale"] = [2.0 ** -6] * G, [2.0 ** -6] * G
        st["out"] = [torch.empty((n * drafts, H, D), dtype=torch.float32, device="cuda") for _ in range(G)]
    if own:
        _own_prepare(st)
    return st


# ---- plain forms ------------------------------------------------------------------------------------------------------------


def _plain_prompt(st):
    """All sequences padded to the longest; scores, softmax and sums in 32 bits."""
    q, k, v = st["q"], st["k"], st["v"]
    n_rows, H, K = q.shape[0], q.shape[1], k.shape[1]
    first, lens = st["row_offset"].long(), st["seq_lens"].long()
    rows = first[1:] - first[:-1]
    i, j = torch.arange(st["max_rows"], device="cuda"), torch.arange(st["max_len"], device="cuda")
    at = (first[:-1, None] + i).clamp(max=n_rows - 1)
    kat = (st["kv_offset"][:, None] + j).clamp(max=k.shape[0] - 1)
    B, N, L, R = at.shape[0], at.shape[1], kat.shape[1], H // K
    qp = q[at].float().view(B, N, K, R, D).permute(0, 2, 3, 1, 4).reshape(B, K, R * N, D)
    s = torch.matmul(qp, k[kat].float().permute(0, 2, 3, 1))
    s.mul_(1.0 / math.sqrt(D))
    seen = (lens - rows)[:, None] + i + 1  # tokens that each row sees
    s.view(B, K, R, N, L).masked_fill_((j >= seen[:, :, None])[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp_(min=-3e38)  # a padded row may see nothing
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v[kat].float().permute(0, 2, 1, 3)).div_(total)
    o = o.view(B, K, R, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, H, D)
    real = i < rows[:, None]
    out = o[real].to(torch.bfloat16)
    if st["lse"] is None:
        return out
    lse = (top + total.log()).view(B, K, R, N).permute(0, 3, 1, 2).reshape(B, N, H)
    return out, lse[real]


def _plain_quantise(x, layer_scale):
    """Codes (two to a byte, the even channel low), group scales (E4M3 bytes) and the values they stand for. In 64 bits:
    a value may lie on the border between two codes."""
    x = x.double().unflatten(-1, (D // GROUP, GROUP))
    top = x.abs().amax(-1)
    fine = torch.isfinite(top)
    want = torch.where(fine, top, 0.0).div(6 * layer_scale).clamp_(max=448)
    _, e = torch.frexp(want)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    s = torch.round(want / step) * step
    use = fine & (s > 0)
    t = x.abs() / torch.where(use, s, 1.0)[..., None] / layer_scale
    code = (t > 0.25).to(torch.uint8) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5)
    code = torch.where(use[..., None], code + 8 * torch.signbit(x).to(torch.uint8), 0).to(torch.uint8).flatten(-2)
    group = torch.where(fine, s.float(), math.nan).to(torch.float8_e4m3fn)
    value = _values(code, group.view(torch.uint8), layer_scale).to(torch.bfloat16)
    return code[..., 0::2] | (code[..., 1::2] << 4), group.view(torch.uint8), value


def _values(code, group, layer_scale):
    """code: one number a byte."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float32, device=code.device)
    table = torch.cat([table, -table])
    scale = group.view(torch.float8_e4m3fn).float() * layer_scale
    return (table[code.long()].unflatten(-1, (D // GROUP, GROUP)) * scale[..., None]).flatten(-2)


def _plain_store(st):
    first, lens = st["row_offset"].long(), st["seq_lens"].long()
    rows = first[1:] - first[:-1]
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), rows, output_size=st["n_rows"])
    at = torch.arange(st["n_rows"], device="cuda") - first[seq] + (st["kv_offset"] + lens - rows)[seq]
    for g in range(len(st["k"])):
        for c in ("k", "v"):
            codes, group, st[c + "_round"][g] = _plain_quantise(st[c + "_new"][g], st[c + "_scale"][g])
            st[c][g][at], st[c + "_group"][g][at] = codes, group
    return _store_outputs(st)


def _store_outputs(st):
    """The caches as they lie in memory, and the new rows' values as the caches now hold them."""
    f8 = lambda xs: [x.view(torch.float8_e4m3fn) for x in xs]
    return dict(k=st["k"], v=st["v"], k_group=f8(st["k_group"]), v_group=f8(st["v_group"]), k_round=st["k_round"],
                v_round=st["v_round"])


def _plain_attend_fp4(st):
    sets = st["sets"].long()
    at = sets.clamp(min=0) + st["kv_offset"][st["q_seq"].long()][:, None]
    out = []
    for g, q in enumerate(st["q"]):
        n, H, K = q.shape[0], q.shape[1], st["k"][g].shape[1]
        kv = []
        for c in ("k", "v"):
            b = st[c][g][at]
            code = torch.stack([b & 15, b >> 4], -1).flatten(-2)
            kv.append(_values(code, st[c + "_group"][g][at], st[c + "_scale"][g]))
        s = torch.matmul(q.float().view(n, K, H // K, D), kv[0].permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D))
        s.masked_fill_((sets < 0)[:, None, None], -math.inf)
        p = (s - s.amax(-1, keepdim=True)).exp_()
        out.append(torch.matmul(p, kv[1].permute(0, 2, 1, 3)).div_(p.sum(-1, keepdim=True)).view(n, H, D))
    return out


# ---- the framework's calls ----------------------------------------------------------------------------------------------------


def _own_prepare(st):
    """What a serving program keeps beside its buffers: the batch descriptor and the workspace."""
    from long_context_sparse_lsa_b200 import binding as lsa

    case = st["case"]
    size = 0
    if case["op"] == "attend_fp4":
        st["batch"] = lsa.Batch(st["kv_offset"], st["seq_lens"], st["q_seq"], st["q_len"], st["max_len"], st["tokens"])
        size = lsa.lsa_attend_fp4_workspace_size(st["batch"], case["heads"], case["kv_heads"], D, st["sets"].shape[1],
                                                 case["layers"])
    else:
        st["prompts"] = lsa.Prompts(st["row_offset"], st["kv_offset"], st["seq_lens"], st["n_rows"], st["max_len"],
                                    st["tokens"])
        if case["op"] == "prompt":
            size = lsa.lsa_attend_prompt_workspace_size(st["prompts"], case["heads"], case["kv_heads"], D)
    st["workspace"] = torch.empty(max(256, size), dtype=torch.uint8, device="cuda")
    st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def _own_run(st):
    from long_context_sparse_lsa_b200 import binding as lsa

    op = st["case"]["op"]
    if op == "prompt":
        lsa.lsa_attend_prompt(st["q"], st["k"], st["v"], st["prompts"], st["out"], st["workspace"], lse=st["lse"],
                              dev_status=st["status"])
        return st["out"] if st["lse"] is None else (st["out"], st["lse"])
    if op == "store":
        lsa.lsa_store_fp4(st["k_new"], st["v_new"], st["k"], st["k_group"], st["v"], st["v_group"], st["k_scale"],
                          st["v_scale"], st["prompts"], k_round=st["k_round"], v_round=st["v_round"],
                          dev_status=st["status"])
        return _store_outputs(st)
    lsa.lsa_attend_fp4(st["q"], st["k"], st["k_group"], st["v"], st["v_group"], st["k_scale"], st["v_scale"], st["sets"],
                       st["batch"], st["out"], st["workspace"], st["status"])
    return st["out"]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    return (_plain_prompt if op == "prompt" else _plain_store if op == "store" else _plain_attend_fp4)(state)


# ---- work and exact values ------------------------------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "attend_fp4":
        budget = case["sink"] + case["window"] + case["topk"]
        lens, G = _contexts(case), case["layers"]
        n = len(lens) * case["drafts"]
        entries = sum(min(budget, x) for x in lens) * case["drafts"]  # each row's tokens, K and V, codes and scales
        row = case["kv_heads"] * (D // 2 + D // GROUP)
        return dict(bytes=G * (2 * entries * row + n * case["heads"] * D * (2 + 4)) + n * budget * 4,
                    flops=4 * G * entries * case["heads"] * D)
    rows, cache = _lengths(case)
    n = sum(rows)
    if op == "prompt":
        H, K = case["heads"], case["kv_heads"]
        pairs = sum(r * c + r * (r + 1) // 2 for r, c in zip(rows, cache))
        return dict(bytes=2 * 2 * n * H * D + 2 * 2 * (n + sum(cache)) * K * D + (4 * n * H if case["lse"] else 0),
                    flops=4 * pairs * H * D)
    each = n * case["kv_heads"] * case["layers"] * 2  # K and V rows: read, codes, scales, the values held
    return dict(bytes=each * (2 * D + D // 2 + D // GROUP + 2 * D), flops=4 * each * D)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "prompt":
        return _exact_prompt(st)
    if op == "store":
        return _exact_store(st)
    return _exact_attend_fp4(st)


def _exact_prompt(st):
    """One sequence and one kv head after the other, at most 4096 rows at a time."""
    case, q, k, v = st["case"], st["q"], st["k"], st["v"]
    H, K = case["heads"], case["kv_heads"]
    R = H // K
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    rows, cache = _lengths(case)
    r0 = c0 = 0
    for n, c in zip(rows, cache):
        for h in range(K):
            for lo in range(0, n, 4096):
                hi = min(n, lo + 4096)
                kk, vv = (x[c0:c0 + c + hi, h].double() for x in (k, v))
                z = torch.einsum("rhd,td->hrt", q[r0 + lo:r0 + hi, h * R:(h + 1) * R].double(), kk) / math.sqrt(D)
                later = torch.ones((hi - lo, c + hi), dtype=torch.bool, device="cuda").triu(c + lo + 1)
                z.masked_fill_(later, -math.inf)
                w = torch.logsumexp(z, -1)
                z.sub_(w[..., None]).exp_()
                out[r0 + lo:r0 + hi, h * R:(h + 1) * R] = torch.einsum("hrt,td->rhd", z, vv)
                lse[r0 + lo:r0 + hi, h * R:(h + 1) * R] = w.T
        r0, c0 = r0 + n, c0 + c + n
    return out if st["lse"] is None else (out, lse)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest(x, values):
    """Index of the value nearest to each x >= 0 (ascending values; of two as near the one with the even index)."""
    v = torch.tensor(values, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(v, x).clamp_(1, len(values) - 1)
    up, down = v[hi] - x, x - v[hi - 1]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def _exact_store(st):
    case = st["case"]
    # E4M3's values from 0 to 448, in the order of their codes 0 .. 126
    e4m3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]
    rows, cache = _lengths(case)
    at, c0 = [], 0
    for n, c in zip(rows, cache):
        at.append(torch.arange(c0 + c, c0 + c + n, device="cuda"))
        c0 += n + c
    at = torch.cat(at)
    got = {n: [] for n in ("k", "v", "k_group", "v_group", "k_round", "v_round")}
    for c in ("k", "v"):
        for x, S in zip(st[c + "_new"], st[c + "_scale"]):
            x = x.double().view(*x.shape[:2], D // GROUP, GROUP)
            byte = _nearest(x.abs().amax(-1) / (6 * S), e4m3)
            s = torch.tensor(e4m3, dtype=torch.float64, device="cuda")[byte]
            code = _nearest(x.abs() / (s * S).clamp(min=1e-300)[..., None], _E2M1)
            value = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")[code] * torch.sign(x) * (s * S)[..., None]
            group = torch.zeros((st["tokens"], x.shape[1], D // GROUP), dtype=torch.float64, device="cuda")
            group[at] = s
            got[c].append(None)  # bytes: the values are in *_group and *_round
            got[c + "_group"].append(group)
            got[c + "_round"].append(value.flatten(-2))
    return got


def _exact_attend_fp4(st):
    """One row after the other."""
    case = st["case"]
    K, R = case["kv_heads"], case["heads"] // case["kv_heads"]
    signed = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device="cuda")
    first = st["kv_offset"].tolist()
    out = []
    for g, q in enumerate(st["q"]):
        o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        for r in range(q.shape[0]):
            e = st["sets"][r]
            at = e[e >= 0].long() + first[int(st["q_seq"][r])]
            kv = []
            for c in ("k", "v"):
                b = st[c][g][at].int()
                x = torch.empty((len(at), K, D), dtype=torch.float64, device="cuda")
                x[..., 0::2], x[..., 1::2] = signed[b % 16], signed[b // 16]
                scale = st[c + "_group"][g][at].view(torch.float8_e4m3fn).double() * st[c + "_scale"][g]
                kv.append(x * scale.repeat_interleave(GROUP, -1))
            z = torch.einsum("hrd,thd->hrt", q[r].double().view(K, R, D), kv[0]) / math.sqrt(D)
            o[r] = torch.einsum("hrt,thd->hrd", torch.softmax(z, -1), kv[1]).reshape(K * R, D)
        out.append(o)
    return out
