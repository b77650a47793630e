"""lsa_attend_prompt on the GPU against softmax(q k^T / sqrt(d)) v in 64 bits.

Tolerance, relative to the largest |V| that a row sees: a weight is rounded to bf16 (half a step, 2^-9 .. 2^-8 of itself), so
that a mean of V rows moves by at most 2^-8 of the largest; the output's own rounding is 2^-8 of it at most (bf16 eps / 2);
fp32 sums and ex2 are far below: 2^-7 together. Errors of single weights are independent, so the relative 2-norm stays below
2^-8 / sqrt(3) for one weight and the output's 2^-8 / sqrt(3): 2^-8 together (sqrt(2 / 3) of 2^-8).
The log-sum-exp is fp32: its sum's relative error (ex2: 2^-22, 128-key partial sums, the scores' 2^-24 * 128 * ~4) is below
2^-15 and so its absolute error, plus 2^-23 of itself.
"""
import numpy as np
import pytest
import torch

from long_context_sparse_lsa_b200 import binding as lsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
MAX, L2, LSE = 2.0 ** -7, 2.0 ** -8, 2.0 ** -15


def _rand(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


class Case:
    def __init__(self, H, K, rows, lens, seed=0, gap=0, fused=False, scale=1.0, max_len=None):
        ro, ko = [0], [gap]
        for n, length in zip(rows, lens):
            ro.append(ro[-1] + n)
            ko.append(ko[-1] + length + gap)
        self.H, self.K, self.rows, self.lens, self.ko, self.ro = H, K, rows, lens, ko[:-1], ro
        self.n, self.total = ro[-1], ko[-1]
        if fused:  # rows of one projection: Q, K, V and something else side by side
            x = _rand((self.n, H + 2 * K + 1, 128), seed)
            self.q, self.k, self.v = x[:, :H], x[:, H:H + K], x[:, H + K:H + 2 * K]
        else:
            self.q, self.k, self.v = (_rand((m, h, 128), seed + i) for i, (m, h) in
                                      enumerate(((self.n, H), (self.total, K), (self.total, K))))
        if scale != 1.0:
            self.q.mul_(scale)
        i32, i64 = (lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)), (lambda x: torch.tensor(x, dtype=torch.int64, device=DEV))
        self.pr = lsa.Prompts(i32(ro), i64(ko[:-1]), i32(lens), self.n, max_len or max(max(lens), 1), self.total)
        self.out = torch.full((self.n, H, 128), 9.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.n, H), 9.0, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        size = lsa.lsa_attend_prompt_workspace_size(self.pr, H, K, 128)
        self.ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device=DEV)

    def run(self, stream=None, lse=True):
        lsa.lsa_attend_prompt(self.q, self.k, self.v, self.pr, self.out, self.ws, self.lse if lse else None, self.status,
                              stream)
        return self

    def want(self, b):
        """Output and log-sum-exp of sequence b's rows in 64 bits, and the largest |V| each row sees."""
        n, length, o = self.rows[b], self.lens[b], self.ko[b]
        q = self.q[self.ro[b]:self.ro[b] + n].double()
        k, v = (x[o:o + length].double() for x in (self.k, self.v))
        R = self.H // self.K
        z = torch.einsum("rhd,thd->hrt", q, k.repeat_interleave(R, 1)) / 128 ** 0.5
        hidden = torch.arange(length, device=DEV) > torch.arange(length - n, length, device=DEV)[:, None]
        z.masked_fill_(hidden, -torch.inf)
        lse = torch.logsumexp(z, -1)
        p = torch.exp(z - lse[..., None])
        # (a weight of 0 times a hidden V that is not finite is not part of the sum)
        out = torch.empty_like(q)
        clean = torch.nan_to_num(v, 0.0, 0.0, 0.0)
        out = torch.einsum("hrt,thd->rhd", p, clean.repeat_interleave(R, 1))
        for t, h, d in (~torch.isfinite(v)).nonzero().tolist():
            first = max(0, t - (length - n))
            out[first:, h * R:(h + 1) * R, d] += v[t, h, d]
        return out, lse.T, float(clean.abs().max())

    def check(self, skip=()):
        assert self.status.item() == 0
        for b, n in enumerate(self.rows):
            if n == 0 or b in skip:
                continue
            want, lse, top = self.want(b)
            got = self.out[self.ro[b]:self.ro[b] + n].double()
            assert torch.equal(got.isnan(), want.isnan()), b
            inf = want.isinf()
            assert torch.equal(got[inf], want[inf]) and torch.equal(got.isinf(), inf), b
            fine = want.isfinite()
            diff = torch.where(fine, got - want, 0.0)
            assert diff.abs().max() <= MAX * top, (b, float(diff.abs().max() / top))
            ref = torch.where(fine, want, 0.0).norm()
            assert diff.norm() <= L2 * ref, (b, float(diff.norm() / ref))
            got_lse = self.lse[self.ro[b]:self.ro[b] + n].double()
            assert torch.equal(got_lse.isnan(), lse.isnan())
            assert (got_lse - lse).nan_to_num().abs().max() <= LSE + 2.0 ** -23 * lse.nan_to_num().abs().max(), b


@pytest.mark.parametrize("H,K", [(1, 1), (8, 1), (16, 1), (4, 2), (32, 4), (4, 4), (6, 2), (5, 1), (28, 4), (64, 1), (12, 1)])
def test_heads(H, K):
    """Groups of 1 to 64 query heads, also ones that do not divide a tile."""
    Case(H, K, [1, 2, 33, 129, 300], [1, 2, 33, 129, 300], seed=H + K).run().check()


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 511, 513, 1000])
@pytest.mark.parametrize("H,K", [(8, 1), (2, 2)])
def test_lengths(n, H, K):
    Case(H, K, [n], [n], seed=n).run().check()


@pytest.mark.parametrize("rows,lens", [
    ([1] * 16, [3136 - 190 * i for i in range(16)]),           # one token each over ragged caches
    ([1], [20000]), ([1], [1]), ([3], [5000]),                   # few rows, long caches: the keys are split
    ([100, 0, 1, 64, 0], [700, 50, 1000, 64, 0]),                # sequences without rows, chunks, a whole prompt
    ([513], [2000]), ([40] * 40, [40 + 13 * i for i in range(40)]),
    ([1] * 1100, [1 + i % 7 for i in range(1100)]),              # more sequences than one search step holds
])
@pytest.mark.parametrize("gap", [0, 5])
def test_caches(rows, lens, gap):
    c = Case(8, 2, rows, lens, seed=len(rows), gap=gap)
    c.run().check()
    c.out.fill_(9.0)
    c.run(lse=False).check()


def test_long_prompt():
    c = Case(8, 2, [5000], [5000], seed=3)
    c.run().check()


@pytest.mark.parametrize("rows,lens", [([70, 300, 1], [70, 300, 1]), ([2048], [2048])])
def test_views_of_a_fused_projection(rows, lens):
    Case(8, 2, rows, lens, fused=True, seed=9).run().check()


@pytest.mark.parametrize("scale", [0.0, 30.0])
def test_flat_and_peaked_softmax(scale):
    """Equal scores, and scores that differ by hundreds (the running maximum moves often)."""
    c = Case(8, 1, [700, 40], [700, 900], scale=scale or 1.0, seed=4)
    if scale == 0.0:
        c.q.zero_()
    else:
        c.k[:900] *= torch.linspace(0.1, 3, 900, device=DEV).to(torch.bfloat16)[:, None, None]  # later keys score higher
    c.run()
    if scale == 30.0:  # scores of size 1000 carry 2^-24 * 1000 * 8 in fp32: 2^-11 of a weight, still below its bf16 rounding
        c.lse.copy_(torch.cat([c.want(b)[1] for b in range(2)]))
    c.check()


def test_rows_behind_and_other_sequences_hold_anything():
    """Cache rows of no sequence hold NaN and infinities; rows of no sequence are left as they were."""
    c = Case(8, 2, [100, 30, 257], [100, 95, 300], gap=200, seed=5)
    used = torch.zeros(c.total, dtype=torch.bool, device=DEV)
    for o, length in zip(c.ko, c.lens):
        used[o:o + length] = True
    c.k[~used] = float("nan")
    c.v[~used] = float("inf")
    c.run().check()
    full = c.out.clone()
    c.pr = lsa.Prompts(c.pr.row_offset[1:3].contiguous(), c.pr.kv_offset[1:2].contiguous(), c.pr.seq_lens[1:2].contiguous(),
                       c.n, c.pr.max_len, c.total)
    c.ws = torch.empty(max(256, lsa.lsa_attend_prompt_workspace_size(c.pr, 8, 2, 128)), dtype=torch.uint8, device=DEV)
    c.out.fill_(9.0)
    c.lse.fill_(9.0)
    c.run()
    assert (c.out[:100] == 9).all() and (c.out[130:] == 9).all() and (c.lse[:100] == 9).all() and (c.lse[130:] == 9).all()
    assert (c.out[100:130].double() - full[100:130].double()).abs().max() <= 2 * MAX * 5


@pytest.mark.parametrize("H,K,n,length", [(8, 1, 300, 300), (1, 1, 700, 800), (8, 1, 1, 4000), (64, 1, 9, 200),
                                          (4, 1, 3, 200), (1, 1, 16, 30), (2, 1, 8, 2500)])
def test_not_finite_where_it_is_seen(H, K, n, length):
    """A K or V that is not finite reaches the rows that see it and no other."""
    for where in (length - 1, max(0, length - n // 2 - 1), length - n):
        c = Case(H, K, [n, 20], [length, 20], seed=6)
        c.v[where, 0, 5], c.v[where, 0, 77], c.v[where, 0, 127] = float("inf"), float("nan"), float("-inf")
        c.run().check()
        c = Case(H, K, [n, 20], [length, 20], seed=7)
        c.k[where, 0, 5] = float("nan")
        c.run().check()
    c = Case(H, K, [n, 20], [length, 20], seed=8)
    c.q[n - 1, 0, 3] = float("nan")
    c.run().check()


@pytest.mark.parametrize("bad", ["rows", "cache", "negative", "max_len", "end"])
@pytest.mark.parametrize("split", [False, True])
def test_bad_sequences_are_skipped(bad, split):
    long = 3000 if split else 60
    c = Case(8, 1, [20, 30, 40] if not split else [1, 2, 1], [50, long, 45], seed=10)
    pr, skip = c.pr, 1
    if bad == "rows":
        pr.seq_lens[1] = c.rows[1] - 1
    elif bad == "cache":
        pr.kv_offset[1] = c.total - long + 1
    elif bad == "negative":
        pr.kv_offset[1] = -1
    elif bad == "max_len":
        pr.seq_lens[1] = pr.max_len + 1
        pr.total_tokens += 0
    else:
        pr.row_offset[3] += 1
        skip = 2
    c.run()
    assert c.status.item() == lsa.LSA_DEV_BAD_LENGTH
    lo, hi = c.ro[skip], c.ro[skip + 1]
    assert (c.out[lo:hi] == 9).all() and (c.lse[lo:hi] == 9).all()
    c.status.zero_()
    c.check(skip=(skip,))


def test_streams_graphs_and_two_calls_at_once():
    a, b = Case(8, 2, [600], [600], seed=1), Case(8, 2, [2], [6000], seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(s1)
        b.run(s2)
    torch.cuda.synchronize()
    a.check()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        b.run()
        a.run()
    for seed in (5, 6):
        a.q.copy_(_rand((600, 8, 128), seed))
        b.v.copy_(_rand((6000, 2, 128), seed))
        graph.replay()
        torch.cuda.synchronize()
        a.check()
        b.check()


def test_same_bits_every_time():
    for rows, lens in (([700, 300], [700, 900]), ([1, 1], [5000, 4000])):
        c = Case(8, 2, rows, lens).run()
        first, lse = c.out.clone(), c.lse.clone()
        for _ in range(5):
            c.run()
            assert torch.equal(c.out, first) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("H,K", [(8, 1), (16, 1), (32, 4), (4, 4), (6, 2), (64, 1), (40, 2)])
@pytest.mark.parametrize("rows,lens", [([1] * 5, [1, 2, 17, 640, 3001]), ([2, 1, 0, 1], [2, 900, 40, 64]), ([1, 40, 1, 1], [700, 100, 65, 64]),
                                       ([1] * 70, [64 + 9 * i for i in range(70)]), ([1, 1, 2], [1000, 3, 129]), ([3, 0], [1500, 0])])
def test_a_token_or_two(H, K, rows, lens):
    """Single tokens, a few of them, and among them a sequence of many."""
    Case(H, K, rows, lens, seed=H, gap=3).run().check()


@pytest.mark.parametrize("rows,lens", [([300, 40], [300, 2000]), ([1, 1], [3000, 2000]), ([1, 1], [900, 600]), ([100], [5000]), ([20], [5000])])
def test_changed_lengths_in_a_captured_call(rows, lens):
    """A graph whose row offsets, lengths and contents change between replays (within max_len), and whose workspace
    another captured call uses too: longer and shorter sequences, rows that move from one to the other, none at all."""
    c = Case(8, 2, rows, lens, seed=5, max_len=max(lens) + 900)
    other = Case(8, 2, [1], [4000], seed=6)
    if other.ws.numel() > c.ws.numel():
        c.ws = torch.empty_like(other.ws)
    other.ws = c.ws
    c.run()
    other.run()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        c.run()
    with torch.cuda.graph(g2, capture_error_mode="thread_local"):
        other.run()
    n, b = c.n, len(rows)
    for new_rows, new_lens in ((rows, lens), ([n] + [0] * (b - 1), [lens[0]] + [0] * (b - 1)),
                               ([n - (b - 1)] + [1] * (b - 1), [max(lens[0] - 700, n)] + [1] * (b - 1)),
                               ([0] * b, [0] * b)):
        c.rows, c.lens = new_rows, new_lens
        c.ro = np.concatenate([[0], np.cumsum(new_rows)]).tolist()
        for t, x in ((c.pr.row_offset, c.ro), (c.pr.seq_lens, new_lens)):
            t.copy_(torch.tensor(x, dtype=torch.int32, device=DEV))
        c.q.copy_(_rand((n, 8, 128), sum(new_lens)))
        c.out.fill_(9.0)
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        skip = [i for i, (r, m) in enumerate(zip(new_rows, new_lens)) if r > m]  # more rows than tokens: refused
        assert c.status.item() == (lsa.LSA_DEV_BAD_LENGTH if skip else 0)
        c.status.zero_()
        c.check(skip)
        other.check()
        assert all((c.out[c.ro[i]:c.ro[i + 1]] == 9).all() for i in skip) and (c.out[c.ro[-1]:] == 9).all()


@pytest.mark.parametrize("rows,lens", [([1, 2], [4000, 1500]), ([200, 7], [900, 300]), ([20], [4000])])
def test_far_rows(rows, lens):
    """Cache rows whose offsets pass 2^32 elements."""
    c = Case(8, 4, rows, lens, seed=2).run()
    near, lse = c.out.clone(), c.lse.clone()
    far = (1 << 23) + 77  # 512 elements a row
    T = far + c.total
    for name in ("k", "v"):
        x = torch.zeros((T, 4, 128), dtype=torch.bfloat16, device=DEV)
        x[far:] = getattr(c, name)
        setattr(c, name, x)
    c.pr = lsa.Prompts(c.pr.row_offset, c.pr.kv_offset + far, c.pr.seq_lens, c.n, c.pr.max_len, T)
    c.run()
    assert c.status.item() == 0 and torch.equal(c.out, near) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("rows,lens", [([60, 90, 1], [500, 500, 500]), ([1, 1, 2], [800, 800, 801])])
def test_sequences_over_the_same_tokens(rows, lens):
    """Sequences that share one cache range."""
    c = Case(8, 2, rows, lens, seed=3)
    c.pr.kv_offset.zero_()
    c.ko = [0] * len(rows)
    c.run().check()


@pytest.mark.parametrize("H,K,rows,lens,max_len", [
    (4096, 64, [3, 1], [3, 40], None), (4096, 64, [1], [300], None), (256, 256, [5], [70], None),
    (8, 1, [40, 3], [40, 90], 1 << 20), (8, 1, [1, 1], [5, 90], 1 << 20), (8, 1, [20], [200], 1 << 20),  # a loose bound
])
def test_extents(H, K, rows, lens, max_len):
    Case(H, K, rows, lens, seed=1, max_len=max_len).run().check()


def test_more_sequences_than_a_grid_axis_holds():
    n = 70000
    c = Case(2, 1, [1] * n, [1 + i % 3 for i in range(n)], seed=4).run()
    assert c.status.item() == 0
    lens, ko = np.array(c.lens), np.array(c.ko)
    k, v = (torch.zeros((n, 3, 128), dtype=torch.float64, device=DEV) for _ in range(2))
    seen = torch.tensor(np.arange(3)[None] < lens[:, None], device=DEV)
    at = torch.tensor(np.minimum(ko[:, None] + np.arange(3)[None], c.total - 1), device=DEV)
    k[seen], v[seen] = c.k[:, 0][at[seen]].double(), c.v[:, 0][at[seen]].double()
    z = torch.einsum("nhd,ntd->nht", c.q.double(), k) / 128 ** 0.5
    p = torch.softmax(z.masked_fill(~seen[:, None], -torch.inf), -1)
    err = (c.out.double() - torch.einsum("nht,ntd->nhd", p, v)).abs().amax((1, 2))
    assert (err <= MAX * v.abs().amax((1, 2))).all()


@pytest.mark.parametrize("H,K,rows,lens", [(4, 1, [3, 1, 1], [200, 5, 70]), (1, 1, [16, 1, 2], [30, 40, 9]), (2, 1, [8, 1], [2500, 30]),
                                           (16, 2, [2, 2, 1], [900, 2, 600])])
def test_not_finite_with_a_few_rows(H, K, rows, lens):
    n, length, h = rows[0], lens[0], H // K
    for where in (length - 1, length - n // 2, length - n, length - n - 1):
        c = Case(H, K, rows, lens, seed=6, gap=2)
        at = c.ko[0] + where
        c.v[at, 0, 5], c.v[at, 0, 77], c.v[at, 0, 127] = float("inf"), float("nan"), float("-inf")
        c.v[c.ko[0] + length:c.ko[0] + length + 2] = float("nan")  # behind the sequence: of nobody
        c.run().check()
        c = Case(H, K, rows, lens, seed=7)
        c.k[where, 0, 5] = float("nan")
        c.run().check()
    c = Case(H, K, rows, lens, seed=8)
    c.q[n - 1, 0, 3] = float("nan")
    c.run().check()
    assert c.out[n - 1, :h].isnan().any()


@pytest.mark.parametrize("H,K,n,length", [(8, 1, 2, 40), (1, 1, 16, 64), (2, 1, 8, 1500), (1, 1, 9, 2000)])
def test_every_new_element_not_finite_with_a_few_rows(H, K, n, length):
    """The V rows of all new tokens but the first hold infinities in every channel: the lanes of a warp zero each other's
    operands, and no row before a token may see 0 times its infinity."""
    c = Case(H, K, [n, 1], [length, 33], seed=11)
    new = torch.arange(length - n + 1, length, device=DEV)
    c.v[c.ko[0] + new] = torch.where(torch.arange(128, device=DEV) % 2 == 0, torch.inf, -torch.inf).to(torch.bfloat16)
    first = None
    for _ in range(20):
        c.out.fill_(9.0)
        c.run()
        assert c.out[0].isfinite().all()  # the first new row sees none of them
        assert c.out[1:n, :, 0::2].eq(torch.inf).all() and c.out[1:n, :, 1::2].eq(-torch.inf).all()
        first = c.out.clone() if first is None else first
        assert torch.equal(c.out, first)
    c.check()


@pytest.mark.parametrize("where", ["behind", "far behind", "before", "far before"])
@pytest.mark.parametrize("rows", [[20, 30, 40, 9], [1, 2, 1, 1], [300, 0, 100, 2000]])
def test_sequences_that_lie_outside_the_rows(where, rows):
    """A sequence none of whose rows lies in the buffers is flagged like one that passes their end."""
    c = Case(8, 1, rows, [max(n, 50) for n in rows], seed=12)
    out = 3 if "behind" in where else 0
    far = 1 << 20 if "far" in where else 0
    if out == 3:  # the last sequence starts at the end of the rows, or far behind
        c.n -= rows[3]
        c.pr.row_offset[3 if far else 4] += far
        c.pr.row_offset[4] += far if far else 0
    else:  # the first one lies before them
        c.n -= rows[0]
        c.ro = [x - rows[0] for x in c.ro]
        c.pr.row_offset -= rows[0]
        c.pr.row_offset[0] -= far
        c.pr.seq_lens[0] += far
        c.pr.max_len += far
    lo = 0 if out == 3 else rows[0]
    c.q, c.out, c.lse = (x[lo:lo + c.n].contiguous() for x in (c.q, c.out, c.lse))
    c.pr.n_rows = c.n
    c.ws = torch.empty(max(256, lsa.lsa_attend_prompt_workspace_size(c.pr, 8, 1, 128)), dtype=torch.uint8, device=DEV)
    c.run()
    assert c.status.item() == lsa.LSA_DEV_BAD_LENGTH
    c.status.zero_()
    skip = [out] + ([2] if out == 3 and far else [])  # (far behind, the sequence before passes the end of the rows)
    c.check(skip=skip)
    for b in skip:
        if b != out:
            assert (c.out[c.ro[b]:c.ro[b + 1]] == 9).all()


@pytest.mark.parametrize("H,K", [(8, 1), (32, 4), (2, 2), (6, 2)])
@pytest.mark.parametrize("many,long", [(3, [3]), (15, [17]), (63, [40, 2, 25]), (700, [256, 5, 300]), (9000, [129, 400, 7])])
def test_chunks_among_single_tokens(H, K, many, long):
    """Single tokens, and a few sequences with many more (row, head) columns than the mean that chooses the kernel."""
    rows = [1] * many
    for i, n in enumerate(long):  # somewhere, and the last at the end
        rows.insert(len(rows) if i + 1 == len(long) else (i + 1) * many // 3, n)
    big = [i for i, n in enumerate(rows) if n > 1]
    lens = [max(n, 1 + (37 * i) % (300 if many < 500 else 20)) for i, n in enumerate(rows)]
    for i in big:
        lens[i] = rows[i] + 500
    c = Case(H, K, rows, lens, seed=many, gap=1).run()
    c.check(skip=() if many < 100 else set(range(len(rows))) - set(big) - set(range(0, len(rows), many // 25)))


def test_a_chunk_in_one_of_many_slots_takes_no_pass_after_pass():
    """64 slots, 63 of them empty, one of 64 rows on 16384 tokens, against the same chunk alone: the mean chooses the kernel
    for a few rows, whose passes over K and V for 16 columns each must not follow one another on a few CTAs (93 times the
    chunk alone, and 7 times now)."""
    def ms(c):
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        times = []
        for _ in range(8):
            ev[0].record()
            c.run()
            ev[1].record()
            torch.cuda.synchronize()
            times.append(ev[0].elapsed_time(ev[1]))
        return sorted(times)[3]

    slots, alone = Case(32, 4, [64] + [0] * 63, [16384] + [1] * 63), Case(32, 4, [64], [16384])
    assert ms(slots) < 25 * ms(alone)
    slots.check()


@pytest.mark.parametrize("rows,lens", [([100], [700]), ([40, 300], [40, 300]), ([1, 1], [5, 900]), ([1] * 200, [30 + i for i in range(200)])])
def test_no_bound_on_the_lengths(rows, lens):
    Case(8, 1, rows, lens, seed=2, max_len=2 ** 31 - 1).run().check()


@pytest.mark.parametrize("rows,lens", [([700, 40], [700, 900]), ([1, 2], [3000, 900]), ([1, 1], [500, 300]), ([100], [5000]), ([64] * 3, [2000, 64, 900])])
@pytest.mark.parametrize("rising", [False, True])
def test_log_sum_exp_of_large_scores(rows, lens, rising):
    """Scores of hundreds, of random order or rising with the position (the running maximum moves in every tile).

    Tolerance. A log-sum-exp moves by no more than its scores do. A score is a sum of 128 exact products, 16 an instruction:
    each of the 8 instructions aligns 17 terms to the largest and drops what lies below 2^-23 of it, and no term or partial
    sum exceeds S = sum |q_i k_i| / sqrt(d): 8 * 17 * 2^-23 S < 2^-15 S (largest S of the row's keys). Taking z c - m c,
    m c + log2 l and the factor ln 2 rounds numbers of at most |lse|'s or S's size four times: 4 * 2^-23 S. LSE for the sum."""
    c = Case(8, 1, rows, lens, scale=30.0, seed=14)
    if rising:
        for o, length in zip(c.ko, c.lens):
            c.k[o:o + length] *= torch.linspace(0.1, 3, length, device=DEV).to(torch.bfloat16)[:, None, None]
    c.run()
    assert c.status.item() == 0
    for b, n in enumerate(rows):
        lse = c.want(b)[1]
        k = c.k[c.ko[b]:c.ko[b] + lens[b]].double().abs().amax(0)  # of each channel
        S = torch.einsum("rhd,kd->rh", c.q[c.ro[b]:c.ro[b] + n].double().abs(), k) / 128 ** 0.5
        got = c.lse[c.ro[b]:c.ro[b] + n].double()
        assert float(lse.abs().max()) > 80  # (the case is what it says)
        assert ((got - lse).abs() <= LSE + (2.0 ** -15 + 2.0 ** -21) * S).all(), (b, float(((got - lse).abs() / S).max()))


@pytest.mark.parametrize("rows,lens", [([70, 300, 1], [70, 300, 1]), ([1, 2, 1], [700, 90, 3]), ([200], [3000]), ([17] * 3, [500, 17, 90])])
@pytest.mark.parametrize("H,K,pad", [(8, 2, 8), (6, 2, 24), (4, 4, 136), (1, 1, 8)])
def test_rows_apart_by_any_multiple_of_eight(rows, lens, H, K, pad):
    """Row strides that are no whole number of heads, bases that are 16-byte aligned and no more."""
    c = Case(H, K, rows, lens, seed=pad)
    for name in ("q", "k", "v"):
        x = getattr(c, name)
        wide = torch.full((x.shape[0] * (x.shape[1] * 128 + pad) + 8,), float("nan"), dtype=torch.bfloat16, device=DEV)
        y = wide[8:].as_strided(x.shape, (x.shape[1] * 128 + pad, 128, 1), 8)
        y.copy_(x)
        assert y.data_ptr() % 32 == 16
        setattr(c, name, y)
    c.run().check()


@pytest.mark.parametrize("n_seq,G", [(40, 8), (4000, 2)])
def test_row_offsets_that_do_not_ascend_end(n_seq, G):
    """Offsets that go up and down name the same rows over and over: the call ends after no more runs of columns than the
    rows can hold. Ones that ascend far behind the rows have no runs."""
    n = 2 * n_seq * 8 // G  # rows that still count as a few per sequence
    c = Case(G, 1, [n] + [0] * (n_seq - 1), [n] + [1] * (n_seq - 1), seed=1)
    c.pr.row_offset.copy_(torch.tensor([0, n] * n_seq, dtype=torch.int32, device=DEV)[:n_seq + 1])
    c.pr.kv_offset.zero_()
    c.pr.seq_lens.fill_(n)
    c.run()
    torch.cuda.synchronize()
    up = torch.arange(n_seq, device=DEV) * (1 << 16)  # ascending, far behind the rows
    c.pr.row_offset[1:] = up.to(torch.int32) + n + 1
    c.out.fill_(9.0)
    c.run()
    assert c.status.item() & lsa.LSA_DEV_BAD_LENGTH and (c.out == 9).all()


@pytest.mark.parametrize("n", [65533, 65534, 65535])
def test_sequences_up_to_the_end_of_a_grid_axis(n):
    """Single tokens and, last, a sequence of 70."""
    c = Case(2, 1, [1] * (n - 1) + [70], [1 + i % 3 for i in range(n - 1)] + [90], seed=4).run()
    c.check(skip=set(range(n)) - set(range(0, n, n // 20)) - {n - 1})


@pytest.mark.parametrize("rows,lens", [([40], [300]), ([1, 1], [3000, 50]), ([2, 1], [200, 300]), ([100], [4000])])
@pytest.mark.parametrize("x", [float("inf"), float("-inf")])
def test_infinite_scores(rows, lens, x):
    """A score of +infinity makes its row and head NaN, the log-sum-exp as well; one of -infinity has no weight."""
    c = Case(8, 2, rows, lens, seed=13)
    at = lens[0] - rows[0]  # seen by every row of the first sequence
    c.k[c.ko[0] + at, 0, 7] = x
    c.run()
    assert c.status.item() == 0
    up = c.q[:rows[0], :4, 7].double() * x > 0  # of the heads that read kv head 0
    out, lse = c.out[:rows[0], :4], c.lse[:rows[0], :4]
    assert torch.equal(out.isnan().any(-1), up) and torch.equal(out.isnan().all(-1), up) and torch.equal(lse.isnan(), up)
    q, k, v = c.q[:rows[0]].double(), c.k[c.ko[0]:c.ko[0] + lens[0]].double(), c.v[c.ko[0]:c.ko[0] + lens[0]].double()
    z = torch.einsum("rhd,td->hrt", q[:, :4], k[:, 0]) / 128 ** 0.5
    z[:, :, at] = -torch.inf  # (the rows whose score is +infinity are not compared)
    z.masked_fill_(torch.arange(lens[0], device=DEV) > torch.arange(lens[0] - rows[0], lens[0], device=DEV)[:, None], -torch.inf)
    p = torch.softmax(z, -1)
    want = torch.einsum("hrt,td->rhd", p, v[:, 0])
    fine = ~up
    assert ((out.double() - want)[fine].abs() <= MAX * v.abs().max()).all()
    assert ((lse.double() - torch.logsumexp(z, -1).T)[fine].abs() <= LSE).all()
