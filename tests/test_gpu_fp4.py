"""The 4-bit cache on the GPU: lsa_store_fp4 byte for byte and lsa_attend_fp4 against their definitions in 64 bits
(fp4_plain.py).

Tolerance of the attention, relative to the largest |V| of the row (the output is a mean of V rows): the weights carry the
scores' error, 8 truncated sums of products of total size ~10 in the exponent (8 * 2^-23 * 10 ~ 1e-5), the two-part P
(2^-22) and the sums over at most 260 tiles (260 * 2^-24 ~ 1.6e-5): below 2^-14 together.
"""
import numpy as np
import pytest
import torch

import fp4_plain as fp4
from long_context_sparse_lsa_b200 import binding as lsa

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -14
DEV = "cuda"


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _i64(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def _rand(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def _caches(T, H, G, fill=0xA5):
    new = lambda n: [torch.full((T, H, n), fill, dtype=torch.uint8, device=DEV) for _ in range(G)]
    return new(64), new(8), new(64), new(8)


def _prompts(rows, lens, total, gap=0, max_len=None, n_rows=None):
    ro, ko = [0], [gap]
    for n, length in zip(rows, lens):
        ro.append(ro[-1] + n)
        ko.append(ko[-1] + length + gap)
    return lsa.Prompts(_i32(ro), _i64(ko[:-1]), _i32(lens), ro[-1] if n_rows is None else n_rows,
                       max_len or max(max(lens), 1), total)


def _special(x):
    """Rows with ties, zeros of both signs, groups of one value, subnormals and the largest values."""
    x = x.clone()
    ties = torch.tensor([6, -6, 5, -5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, 0.5, -0.0, 0.0, -1e-30, 1e-30])
    x[0, 0, :16] = ties.to(x)
    x[0, 0, 16:32] = 0
    x[0, 0, 32:48] = -0.0
    x[0, 0, 48:64] = 3e38
    x[0, 0, 64:80] = 1e-39
    x[0, 0, 80:96] = torch.arange(16).to(x) * 2.0 ** -13
    x[0, 0, 96:112] = (ties * 2.0 ** -16).to(x)
    x[0, 0, 112:128] = (ties * 13 / 8).to(x)
    return x


@pytest.mark.parametrize("H,G,rows,lens,scale", [
    (4, 1, [1] * 16, [37 + i for i in range(16)], 1.0),       # a decode step
    (4, 2, [4] * 5, [4, 5, 100, 6, 300], 2.0 ** -6),           # draft tokens; a sequence of new tokens only
    (1, 1, [0, 3, 0, 0, 200, 1, 0], [0, 3, 5, 0, 200, 77, 1], 2.0 ** 3),  # sequences without rows
    (3, 1, [41, 17], [41, 30], 1.0),                           # a token's groups do not divide the CTA's
    (8, 8, [33], [40], 2.0 ** -20),
    (2, 1, [1] * 1100, [2] * 1100, 1.0),                       # more sequences than one search step holds
    (4, 1, [5000], [6000], 2.0 ** -4),
])
@pytest.mark.parametrize("fused", [False, True])
def test_store_bytes(H, G, rows, lens, scale, fused):
    n, gap = sum(rows), 3
    total = sum(lens) + gap * (len(lens) + 1)
    k_sc, v_sc = [scale * 2.0 ** g for g in range(G)], [scale / 2 ** g for g in range(G)]
    k_new, v_new = [], []
    for g in range(G):
        if fused:  # K and V as views of one buffer, one row of which holds both and more
            buf = _rand((n, 2 * H + 1, 128), 7 * g + H)
            buf[:, :H] = _special(buf[:, :H])
            k_new.append(buf[:, :H])
            v_new.append(buf[:, H + 1:])
        else:
            k_new.append(_special(_rand((n, H, 128), 7 * g + H)))
            v_new.append(_rand((n, H, 128), 7 * g + H + 1, 30.0))
    k, kg, v, vg = _caches(total, H, G)
    kr = [torch.empty((n, H, 128), dtype=torch.bfloat16, device=DEV) for _ in range(G)]
    vr = [torch.empty_like(x) for x in kr]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pr = _prompts(rows, lens, total, gap)
    lsa.lsa_store_fp4(k_new, v_new, k, kg, v, vg, k_sc, v_sc, pr, kr, vr, status)
    assert status.item() == 0
    again = _caches(total, H, G)
    lsa.lsa_store_fp4(k_new, v_new, *again, k_sc, v_sc, pr)  # without the rounded rows
    at = np.concatenate([np.arange(o + length - r, o + length) for o, length, r in
                         zip(pr.kv_offset.tolist(), lens, rows)]).astype(int)
    for new, code, group, rnd, sc, code2, group2 in ((k_new, k, kg, kr, k_sc, again[0], again[1]),
                                                     (v_new, v, vg, vr, v_sc, again[2], again[3])):
        for g in range(G):
            wc, wg, wv = fp4.quantise(new[g], sc[g])
            full_c = np.full((total, H, 64), 0xA5, np.uint8)
            full_g = np.full((total, H, 8), 0xA5, np.uint8)
            full_c[at], full_g[at] = wc, wg
            assert np.array_equal(group[g].cpu().numpy(), full_g)
            assert np.array_equal(code[g].cpu().numpy(), full_c)
            assert torch.equal(code[g], code2[g]) and torch.equal(group[g], group2[g])
            want = torch.tensor(wv).to(torch.bfloat16)
            assert torch.equal(rnd[g].cpu(), want)


def test_store_not_finite():
    x = _rand((2, 4, 128), 1)
    x[0, 1, 5], x[0, 2, 17], x[1, 3, 127] = float("nan"), float("inf"), float("-inf")
    k, kg, v, vg = _caches(2, 4, 1)
    kr, vr = [torch.empty_like(x)], [torch.empty_like(x)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lsa.lsa_store_fp4([x], [_rand((2, 4, 128), 2)], k, kg, v, vg, [1.0], [1.0], _prompts([2], [2], 2), kr, vr, status)
    assert status.item() == lsa.LSA_DEV_BAD_VALUE
    wc, wg, wv = fp4.quantise(x, 1.0)
    assert np.array_equal(k[0].cpu().numpy(), wc) and np.array_equal(kg[0].cpu().numpy(), wg)
    assert np.array_equal(np.isnan(kr[0].float().cpu().numpy()), np.isnan(wv)) and np.isnan(wv).sum() == 48


@pytest.mark.parametrize("bad", ["rows", "cache", "negative", "max_len", "end"])
def test_store_skips_bad_sequences(bad):
    """A sequence that does not fit is flagged and skipped, the others are stored."""
    rows, lens, total = [2, 3, 2], [4, 5, 6], 15
    ro, ko, sl, n_rows, max_len = [0, 2, 5, 7], [0, 4, 9], list(lens), 7, 6
    if bad == "rows":
        sl[1] = 2
    elif bad == "cache":
        ko[1] = 11
    elif bad == "negative":
        ko[1] = -1
    elif bad == "max_len":
        sl[1], max_len = 5, 4
        sl[2] = 4
    else:
        ro[3], n_rows = 9, 7  # the last sequence's rows pass the end
    x = _rand((n_rows, 2, 128), 3)
    k, kg, v, vg = _caches(total, 2, 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lsa.lsa_store_fp4([x], [x], k, kg, v, vg, [1.0], [1.0], lsa.Prompts(_i32(ro), _i64(ko), _i32(sl), n_rows, max_len, total),
                      dev_status=status)
    assert status.item() == lsa.LSA_DEV_BAD_LENGTH
    want = np.full((total, 2, 64), 0xA5, np.uint8)
    codes = fp4.quantise(x, 1.0)[0]
    for b in range(3):
        if b != (2 if bad == "end" else 1):
            n = rows[b]
            want[ko[b] + sl[b] - n:ko[b] + sl[b]] = codes[ro[b]:ro[b] + n]
    assert np.array_equal(k[0].cpu().numpy(), want) and np.array_equal(v[0].cpu().numpy(), want)


def test_store_rows_of_no_sequence_are_left():
    x = _rand((10, 1, 128), 4)
    k, kg, v, vg = _caches(20, 1, 1)
    kr, vr = [torch.full_like(x, 7.0)], [torch.full_like(x, 7.0)]
    lsa.lsa_store_fp4([x], [x], k, kg, v, vg, [1.0], [1.0], lsa.Prompts(_i32([2, 4, 7]), _i64([0, 10]), _i32([2, 3]), 10, 20, 20),
                      kr, vr)
    assert (kr[0][:2] == 7).all() and (kr[0][7:] == 7).all() and (k[0][2:10] == 0xA5).all() and (k[0][13:] == 0xA5).all()
    assert np.array_equal(kr[0][2:7].float().cpu().numpy(), fp4.quantise(x, 1.0)[2][2:7])


# ---- attention -------------------------------------------------------------------------------------------------------------


class Case:
    """Rows of one or more sequences over random 4-bit caches."""

    def __init__(self, H, K, G, lens, sets, q_seq, q_len, seed=0, gap=2):
        self.H, self.K, self.G = H, K, G
        off = [gap + i * gap + sum(lens[:i]) for i in range(len(lens))]
        self.off, self.lens, self.q_seq, self.q_len = off, lens, q_seq, q_len
        self.total = off[-1] + lens[-1] + gap
        self.n = len(q_seq)
        self.sets = _i32(sets).reshape(self.n, -1)
        self.q = [_rand((self.n, H, 128), seed + g) for g in range(G)]
        self.k_scale, self.v_scale = [2.0 ** -6 * (g + 1) for g in range(G)], [-0.01 * (g + 1) for g in range(G)]
        self.k, self.kg, self.v, self.vg = [], [], [], []
        for g in range(G):
            for j, (codes, groups) in enumerate(((self.k, self.kg), (self.v, self.vg))):
                c, s, _ = fp4.quantise(_rand((self.total, K, 128), 100 + seed + 2 * g + j), 2.0 ** -6)
                codes.append(torch.tensor(c, device=DEV))
                groups.append(torch.tensor(s, device=DEV))
        self.out = [torch.full((self.n, H, 128), 9.0, device=DEV) for _ in range(G)]
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.batch = lsa.Batch(_i64(off), _i32(lens), _i32(q_seq), _i32(q_len), max(lens), self.total)
        size = lsa.lsa_attend_fp4_workspace_size(self.batch, H, K, 128, self.sets.shape[1], G)
        self.ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device=DEV)  # NaN bits: nothing relies on it

    def run(self, stream=None):
        lsa.lsa_attend_fp4(self.q, self.k, self.kg, self.v, self.vg, self.k_scale, self.v_scale, self.sets, self.batch,
                           self.out, self.ws, self.status, stream)
        return self

    def want(self, g, r):
        o = self.off[self.q_seq[r]]
        span = slice(o, o + self.lens[self.q_seq[r]])
        kv = [fp4.values(c[g][span].cpu().numpy(), s[g][span].cpu().numpy(), sc[g])
              for c, s, sc in ((self.k, self.kg, self.k_scale), (self.v, self.vg, self.v_scale))]
        return fp4.attend(self.q[g][r], kv[0], kv[1], self.sets[r].cpu().numpy()), np.nanmax(np.abs(kv[1]))

    def check(self, rows=None):
        for g in range(self.G):
            for r in rows if rows is not None else range(self.n):
                want, top = self.want(g, r)
                got = self.out[g][r].double().cpu().numpy()
                assert np.array_equal(np.isnan(got), np.isnan(want)), (g, r)
                assert np.nanmax(np.abs(got - want), initial=0.0) <= TOL * top, (g, r)


def _sets(q_len, budget, seed=0):
    rng = np.random.default_rng(seed)
    out = np.full((len(q_len), budget), -1, np.int64)
    for r, length in enumerate(q_len):
        n = min(length, budget)
        out[r, :n] = np.sort(rng.choice(length, n, replace=False))
    return out.tolist()


@pytest.mark.parametrize("H,K", [(1, 1), (8, 1), (16, 1), (4, 2), (32, 4), (4, 4), (8, 8), (64, 4)])
@pytest.mark.parametrize("budget", [1, 16, 57, 400])
def test_attend_heads_and_budgets(H, K, budget):
    lens = [300, 1, 17, 1000]
    q_seq, q_len = [0, 1, 2, 3, 3], [300, 1, 17, 1000, 999]
    c = Case(H, K, 1, lens, _sets(q_len, budget), q_seq, q_len, seed=H + budget).run()
    assert c.status.item() == 0
    c.check()


@pytest.mark.parametrize("n,budget,G", [(1, 3136, 1), (1, 4160, 4), (16, 3136, 2), (150, 388, 1), (2, 16384, 1)])
def test_attend_split_and_whole(n, budget, G):
    """One row over many CTAs, several rows, more rows than SMs, the largest budget."""
    lens = [max(budget + 100, 500)]
    q_len = [lens[0] - i for i in range(n)]
    c = Case(32 if budget < 10000 else 8, 4 if budget < 10000 else 1, G, lens, _sets(q_len, budget), [0] * n, q_len).run()
    assert c.status.item() == 0
    c.check(range(0, n, max(1, n // 5)))


def test_attend_any_set():
    """No entry, holes, entries twice, no order, entries behind the row's length's worth of slots."""
    sets = [[-1] * 40, [-1] * 30 + [4, 4, 4, 2] + [-1] * 6, list(range(39, -1, -1)), [-1] * 39 + [0], [7] * 40]
    c = Case(8, 2, 2, [40], sets, [0] * 5, [40, 5, 40, 1, 8]).run()
    assert c.status.item() == 0
    c.check()
    assert (c.out[0][0] == 0).all()
    empty = Case(8, 2, 1, [40], [[], []], [0, 0], [40, 3]).run()
    assert (empty.out[0] == 0).all() and empty.status.item() == 0


def test_attend_flags_bad_entries_and_rows():
    sets = [[0, 5, 40, -2, 3], [0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [0, 1, 2, 3, 4]]
    c = Case(8, 2, 1, [40, 6], sets, [0, 0, 1, 1, 1], [40, 40, 6, 5, 5])
    c.run()
    assert c.status.item() == lsa.LSA_DEV_BAD_INDEX
    c.sets[0] = _i32([0, 5, 3, -1, -1])  # what is left of the first set
    c.check()
    for q_seq, q_len, bit in [([0, 2, 1, -1, 1], None, lsa.LSA_DEV_BAD_SEQ), (None, [40, 0, 6, 7, 5], lsa.LSA_DEV_BAD_LENGTH)]:
        c.status.zero_()
        c.batch.q_seq = _i32(q_seq or c.q_seq)
        c.batch.q_len = _i32(q_len or c.q_len)
        c.run()
        assert c.status.item() & bit
        c.batch.q_seq, c.batch.q_len = _i32(c.q_seq), _i32(c.q_len)
        c.check([0, 2, 4])
        assert (c.out[0][1] == 0).all() and (c.out[0][3] == 0).all()
        c.out[0].fill_(9.0)


def test_attend_nan_and_large_values():
    """NaN groups count only where they are selected, in V only for their channels; a query of any finite size is taken,
    one that is not finite gives NaN for its head."""
    sets = [list(range(0, 64)), list(range(64, 128)), [70] + [-1] * 63, list(range(0, 64)), list(range(0, 64))]
    c = Case(16, 2, 1, [128], sets, [0] * 5, [128] * 5)
    c.kg[0][c.off[0] + 70, 1, 3] = 0x7F
    c.vg[0][c.off[0] + 71, 0, 2] = 0xFF
    c.q[0][3] *= 2.0 ** 100
    c.k_scale = [2.0 ** -106]  # together the scores of row 3 are of ordinary size, the others' vanish
    c.q[0][4, 3, 9] = float("inf")
    c.q[0][4, 12, 0] = float("nan")
    c.q[0][0, 2] = 0
    c.run()
    c.check()
    out = c.out[0]
    assert not out[[0, 3]].isnan().any() and out[1, 8:].isnan().all() and out[1, :8, 32:48].isnan().all()
    assert out[2, 8:].isnan().all() and not out[2, :8].isnan().any()
    assert out[4, 3].isnan().all() and out[4, 12].isnan().all() and not out[4, 4].isnan().any()


def test_attend_far_rows():
    """Cache rows whose byte offsets pass 2^32."""
    T, K = (1 << 26) // 4 + 5000, 4  # codes: 4.3 GB
    k = torch.zeros((T, K, 64), dtype=torch.uint8, device=DEV)
    v, kg, vg = torch.zeros_like(k), *(torch.zeros((T, K, 8), dtype=torch.uint8, device=DEV) for _ in range(2))
    small = Case(32, 4, 1, [5000], _sets([5000], 600), [0], [5000], gap=0)
    for far, near in ((k, small.k), (kg, small.kg), (v, small.v), (vg, small.vg)):
        far[T - 5000:] = near[0]
    small.run()
    near_out = small.out[0].clone()
    small.k, small.kg, small.v, small.vg = [k], [kg], [v], [vg]
    small.batch = lsa.Batch(_i64([T - 5000]), _i32([5000]), _i32([0]), _i32([5000]), 5000, T)
    small.run()
    assert small.status.item() == 0 and torch.equal(small.out[0], near_out)
    rows = _rand((3, K, 128), 5)
    lsa.lsa_store_fp4([rows], [rows], [k], [kg], [v], [vg], [1.0], [1.0],
                      lsa.Prompts(_i32([0, 3]), _i64([T - 5000]), _i32([5000]), 3, 5000, T))
    assert np.array_equal(k[T - 3:].cpu().numpy(), fp4.quantise(rows, 1.0)[0])


def test_streams_graphs_and_two_calls_at_once():
    a = Case(32, 4, 1, [4000], _sets([4000], 3136), [0], [4000], seed=1)
    b = Case(32, 4, 1, [4000], _sets([4000], 3136, 5), [0], [4000], seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.run(s1)
        b.run(s2)
    torch.cuda.synchronize()
    a.check()
    b.check()
    first = a.out[0].clone()
    new = _rand((1, 4, 128), 9)
    pr = lsa.Prompts(_i32([0, 1]), _i64(a.off), _i32(a.lens), 1, 4000, a.total)
    store = lambda: lsa.lsa_store_fp4([new], [new], a.k, a.kg, a.v, a.vg, [2.0 ** -6], [2.0 ** -6], pr)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        store()
        a.run()
    for seed in (11, 12):  # new contents in the captured buffers
        new.copy_(_rand((1, 4, 128), seed))
        a.sets.copy_(_i32(_sets([4000], 3136, seed)))
        a.sets[0, -1] = 3999  # the stored token is read
        graph.replay()
        torch.cuda.synchronize()
        a.check()
    assert not torch.equal(a.out[0], first)


def test_same_bits_every_time():
    c = Case(32, 4, 2, [5000], _sets([5000] * 3, 3136), [0] * 3, [5000] * 3)
    first = [x.clone() for x in c.run().out]
    for _ in range(5):
        c.run()
        assert all(torch.equal(x, y) for x, y in zip(first, c.out))


def test_store_changed_lengths_in_a_captured_call():
    """A graph whose row offsets and lengths change between replays; rows behind the last sequence are not stored."""
    lens, rows, H = [300, 500], [40, 24], 2
    pr = _prompts(rows, lens, 900, max_len=600)
    new = [_rand((64, H, 128), i) for i in (1, 2)]
    caches = _caches(900, H, 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    store = lambda: lsa.lsa_store_fp4(new[:1], new[1:], *caches, [0.5], [2.0], pr, dev_status=status)
    store()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        store()
    for n_rows, n_lens in (([40, 24], [300, 500]), ([0, 64], [7, 64]), ([1, 1], [1, 600]), ([0, 0], [0, 0])):
        pr.row_offset.copy_(_i32([0, n_rows[0], sum(n_rows)]))
        pr.seq_lens.copy_(_i32(n_lens))
        pr.kv_offset.copy_(_i64([3, 300]))
        for x in caches:
            x[0].fill_(0xA5)
        for i in (0, 1):
            new[i].copy_(_rand((64, H, 128), sum(n_lens) + i))
        graph.replay()
        torch.cuda.synchronize()
        assert status.item() == 0
        at = np.concatenate([np.arange(o + n - r, o + n) for o, n, r in zip((3, 300), n_lens, n_rows)]).astype(int)
        for i, (code, group, sc) in enumerate(((caches[0], caches[1], 0.5), (caches[2], caches[3], 2.0))):
            wc, wg, _ = fp4.quantise(new[i], sc)
            full_c, full_g = np.full((900, H, 64), 0xA5, np.uint8), np.full((900, H, 8), 0xA5, np.uint8)
            full_c[at], full_g[at] = wc[:len(at)], wg[:len(at)]
            assert np.array_equal(code[0].cpu().numpy(), full_c) and np.array_equal(group[0].cpu().numpy(), full_g)


def test_store_every_scale_and_mantissa():
    """Groups whose largest magnitude takes every bf16 mantissa at 60 exponents, with ties and neighbours of every border
    of both roundings among them, byte for byte."""
    m = torch.arange(128, 256, device=DEV, dtype=torch.float64)
    e = torch.arange(-34, 26, device=DEV, dtype=torch.float64)
    top = (m[None] * 2.0 ** e[:, None]).reshape(-1)              # 7680 groups
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    rest = torch.randint(0, 256, (top.numel(), 15), generator=g, device=DEV).double() / 256 * top[:, None]
    rest *= torch.randint(0, 2, rest.shape, generator=g, device=DEV) * 2 - 1
    x = torch.cat([top[:, None], rest], 1).to(torch.bfloat16).view(-1, 4, 128)
    n = x.shape[0]
    for S in (1.0, 2.0 ** -7, 2.0 ** 40, 2.0 ** -40):
        k, kg, v, vg = _caches(n, 4, 1)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        y = -x
        lsa.lsa_store_fp4([x], [y], k, kg, v, vg, [S], [S], _prompts([n], [n], n), dev_status=status)
        assert status.item() == 0
        for new, code, group in ((x, k, kg), (y, v, vg)):
            wc, wg, _ = fp4.quantise(new, S)
            assert np.array_equal(group[0].cpu().numpy(), wg) and np.array_equal(code[0].cpu().numpy(), wc)


@pytest.mark.parametrize("H,G,rows,lens", [(4, 1, [5000, 1, 6999], [5000, 300, 7100]), (3, 2, [4099], [4099]), (256, 1, [301], [400])])
def test_store_many_rows(H, G, rows, lens):
    """Enough rows that a thread takes two groups; a last CTA that is not full."""
    n = sum(rows)
    total = sum(lens) + 4 * (len(lens) + 1)
    pr = _prompts(rows, lens, total, 4)
    k_new, v_new = ([_rand((n, H, 128), 3 * g + i) for g in range(G)] for i in (0, 1))
    scale = [2.0 ** -g for g in range(G)]
    k, kg, v, vg = _caches(total, H, G)
    kr, vr = ([torch.empty((n, H, 128), dtype=torch.bfloat16, device=DEV) for _ in range(G)] for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lsa.lsa_store_fp4(k_new, v_new, k, kg, v, vg, scale, scale, pr, kr, vr, status)
    again = _caches(total, H, G)
    lsa.lsa_store_fp4(k_new, v_new, *again, scale, scale, pr)
    assert status.item() == 0
    at = np.concatenate([np.arange(o + m - r, o + m) for o, m, r in zip(pr.kv_offset.tolist(), lens, rows)]).astype(int)
    for new, code, group, rnd, code2, group2 in ((k_new, k, kg, kr, again[0], again[1]), (v_new, v, vg, vr, again[2], again[3])):
        for g in range(G):
            wc, wg, wv = fp4.quantise(new[g], scale[g])
            full_c, full_g = np.full((total, H, 64), 0xA5, np.uint8), np.full((total, H, 8), 0xA5, np.uint8)
            full_c[at], full_g[at] = wc, wg
            assert np.array_equal(group[g].cpu().numpy(), full_g) and np.array_equal(code[g].cpu().numpy(), full_c)
            assert torch.equal(code[g], code2[g]) and torch.equal(group[g], group2[g])
            assert torch.equal(rnd[g].cpu(), torch.tensor(wv).to(torch.bfloat16))


@pytest.mark.parametrize("ro,here", [([0, 2, 7, 9], (0, 1)), ([0, 2, 7, 5000], (0, 1)), ([0, 2, 100000, 100003], (0,)),
                                     ([-3, 0, 4, 7], (1, 2)), ([-4000, -3995, 0, 7], (2,)), ([7, 9, 10, 12], ())])
def test_store_flags_sequences_outside_the_rows(ro, here):
    """Also one none of whose rows lies in the buffers."""
    n_rows, lens, ko = 7, [8, 8, 8], [0, 8, 16]
    x = _rand((n_rows, 2, 128), 3)
    k, kg, v, vg = _caches(24, 2, 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lsa.lsa_store_fp4([x], [x], k, kg, v, vg, [1.0], [1.0], lsa.Prompts(_i32(ro), _i64(ko), _i32(lens), n_rows, 8, 24),
                      dev_status=status)
    assert status.item() == lsa.LSA_DEV_BAD_LENGTH
    want = np.full((24, 2, 64), 0xA5, np.uint8)
    codes = fp4.quantise(x, 1.0)[0]
    for b in here:
        n = ro[b + 1] - ro[b]
        want[ko[b] + lens[b] - n:ko[b] + lens[b]] = codes[ro[b]:ro[b + 1]]
    assert np.array_equal(k[0].cpu().numpy(), want) and np.array_equal(v[0].cpu().numpy(), want)


@pytest.mark.parametrize("H,K", [(8, 1), (16, 1), (8, 4)])
def test_attend_small_queries(H, K):
    """Query rows around and below the smallest normal bf16, of full weight where the layer's scale is large."""
    c = Case(H, K, 1, [300], _sets([300] * 4, 200), [0] * 4, [300] * 4, seed=H)
    for r, e in enumerate((-124, -127, -130, -133)):
        c.q[0][r] = (c.q[0][r].double() * 2.0 ** e).to(torch.bfloat16)
    c.k_scale = [2.0 ** 120]  # (numbers of size 2^126: scores of size 4 to 2^-7)
    c.run()
    assert c.status.item() == 0 and c.q[0][2].abs().max() > 0
    c.check()


@pytest.mark.parametrize("H,pad", [(2, 8), (3, 40), (1, 136)])
def test_store_rows_apart_by_any_multiple_of_eight(H, pad):
    n = 77
    x = _rand((n, H, 128), pad)
    wide = torch.full((n * (H * 128 + pad) + 8,), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = wide.as_strided(x.shape, (H * 128 + pad, 128, 1), 8)
    y.copy_(x)
    assert y.data_ptr() % 32 == 16
    k, kg, v, vg = _caches(n, H, 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lsa.lsa_store_fp4([y], [x], k, kg, v, vg, [0.5], [0.5], _prompts([n], [n], n), dev_status=status)
    wc, wg, _ = fp4.quantise(x, 0.5)
    assert status.item() == 0 and np.array_equal(k[0].cpu().numpy(), wc) and np.array_equal(kg[0].cpu().numpy(), wg)
    assert torch.equal(k[0], v[0]) and torch.equal(kg[0], vg[0])
