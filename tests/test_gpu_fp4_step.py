"""The 4-bit cache in use: whole prompts attended and stored, their indexer keys summed, decode steps over the cache
(LsaStep), eager and as graphs.

Index sets are compared bit for bit with the oracle's; attention with its definition in 64 bits on the values the cache
holds (test_gpu_fp4.py and test_gpu_prompt.py derive the two tolerances).
"""
import numpy as np
import pytest
import torch

import fp4_plain as fp4
import parity
from long_context_sparse_lsa_b200 import binding as lsa
from long_context_sparse_lsa_b200 import workloads as wls
from long_context_sparse_lsa_b200.pipeline import LsaStep

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -14
DEV = "cuda"
BASE = wls.Workload("fp4", 0, (3000,), 16, 128, -16, 15, 8, 16, 128, 256, 0, 0, 32, 4, 128, 1)


def _cache(st, g, b):
    """Sequence b's K and V of layer g, in 64 bits."""
    o, n = int(st.t.kv_offset[b]), int(st.t.seq_lens[b])
    part = lambda x: x[g][o:o + n].cpu().numpy()
    return (fp4.values(part(st.k4), part(st.k4_group), st.k_scale[g]),
            fp4.values(part(st.v4), part(st.v4_group), st.v_scale[g]))


def _check(st):
    assert st.status_bits() == 0
    want = parity.oracle_sets(st.wl, st.t)
    parity.check_sets(parity.host(st.sets), want, st.wl.name)
    for g in range(st.G):
        for b in range(st.wl.n_seq):
            k, v = _cache(st, g, b)
            for r in (st.t.q_seq == b).nonzero()[:, 0].tolist():
                ref = fp4.attend(st.t.q[g][r], k, v, want[r])
                err = np.abs(st.out[g][r].cpu().numpy() - ref).max()
                assert err <= TOL * np.abs(v).max(), (g, r, err)


def _check_new_rows(st):
    for g in range(st.G):
        for b in range(st.wl.n_seq):
            o, n = int(st.t.kv_offset[b]), int(st.t.seq_lens[b])
            for new, code, group, sc in ((st.k_new, st.k4, st.k4_group, st.k_scale),
                                         (st.v_new, st.v4, st.v4_group, st.v_scale)):
                wc, wg, _ = fp4.quantise(new[g][b], sc[g])
                assert np.array_equal(code[g][o + n - st.n_new:o + n].cpu().numpy(), wc)
                assert np.array_equal(group[g][o + n - st.n_new:o + n].cpu().numpy(), wg)


@pytest.mark.parametrize("kw,fuse", [
    (dict(lens=(3000, 17, 1, 900)), True),
    (dict(lens=(6000, 2500), hi_block=64, hi_topblocks=8, G=3, drafts=3), True),
    (dict(lens=(6000, 2500), hi_block=64, hi_topblocks=8), False),
    (dict(lens=(2000,), prefill_new=37, G=2), True),
    (dict(lens=(1500, 700), H_q=64), True),
    (dict(lens=(500,), H_q=8, H_kv=1, drafts=4), False),
])
def test_step(kw, fuse):
    wl = wls.small(BASE, seed=51, **kw)
    st = LsaStep(wl, wls.make(wl, DEV, with_kv=False), DEV, kv_fp4=True, fuse_append=fuse)
    st.build_block_sums()
    st.step()
    torch.cuda.synchronize()
    _check(st)
    if st.n_new:
        _check_new_rows(st)


def test_graphs_and_new_rows():
    """The captured step on new inputs, and the step with its host copies."""
    wl = wls.small(BASE, lens=(4000, 900), G=2, hi_block=64, hi_topblocks=16, seed=52)
    st = LsaStep(wl, wls.make(wl, DEV, with_kv=False), DEV, kv_fp4=True)
    st.build_block_sums()
    st.pack_io()
    st.capture()
    for seed in (1, 2):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        for x in [*st.k_new, *st.v_new, *st.t.q]:
            x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        st.replay()
        torch.cuda.synchronize()
        _check(st)
        _check_new_rows(st)
    h_in = torch.empty(st.in_buf.numel(), dtype=torch.uint8, pin_memory=True)
    h_out = torch.empty(st.out_buf.numel(), dtype=torch.uint8, pin_memory=True)
    h_in.copy_(st.in_buf)
    want = st.out_buf.clone()
    st.out_buf.zero_()
    st.in_buf.zero_()
    st.capture_e2e(h_in, h_out)
    st.replay("e2e")
    torch.cuda.synchronize()
    assert torch.equal(h_out, want.cpu())


def test_prompts_then_steps():
    """Prompts of two sequences, in two chunks each: attention over bf16 K/V, the rows into the 4-bit cache (taking the
    cache's values for the next chunk), the keys' block sums, then decode steps that append a token at a time."""
    first, second, steps = (700, 129), (400, 1), 3
    lens = tuple(a + b + steps for a, b in zip(first, second))
    wl = wls.small(BASE, lens=lens, hi_block=64, hi_topblocks=4, seed=53)
    t = wls.make(wl, DEV, with_kv=False)
    st = LsaStep(wl, t, DEV, kv_fp4=True)
    T, H, K, d = wl.total_tokens, wl.H_q, wl.H_kv, wl.d
    for x in (*st.k4, *st.v4, *st.k4_group, *st.v4_group):
        x.zero_()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    k_rows, v_rows = (torch.zeros((T, K, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    offs = t.kv_offset.tolist()
    kc, vc = (np.zeros((T, K, d)) for _ in range(2))
    done = [0, 0]
    for chunk in (first, second):
        done = [a + b for a, b in zip(done, chunk)]
        n = sum(chunk)
        pr = lsa.Prompts(i32([0, chunk[0], n]), t.kv_offset, i32(done), n, max(done), T)
        fused = torch.randn((n, H + 2 * K, d), generator=gen, device=DEV).to(torch.bfloat16)
        q, kn, vn = fused[:, :H], fused[:, H:H + K], fused[:, H + K:]
        at = torch.cat([torch.arange(o + e - c, o + e) for o, e, c in zip(offs, done, chunk)]).to(DEV)
        # later chunks see what the cache holds: the rounded rows
        rk, rv = [torch.empty((n, K, d), dtype=torch.bfloat16, device=DEV)], [torch.empty((n, K, d), dtype=torch.bfloat16, device=DEV)]
        lsa.lsa_store_fp4([kn], [vn], st.k4, st.k4_group, st.v4, st.v4_group, st.k_scale, st.v_scale, pr, rk, rv, st.status)
        k_rows[at], v_rows[at] = rk[0], rv[0]
        out = torch.empty((n, H, d), dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(max(1, lsa.lsa_attend_prompt_workspace_size(pr, H, K, d)), dtype=torch.uint8, device=DEV)
        lsa.lsa_attend_prompt(q, k_rows, v_rows, pr, out, ws, None, st.status)
        torch.cuda.synchronize()
        a = at.cpu().numpy()
        kc[a], vc[a] = fp4.quantise(kn, st.k_scale[0])[2], fp4.quantise(vn, st.v_scale[0])[2]
        row = 0
        for b, (o, e, c) in enumerate(zip(offs, done, chunk)):
            for i in range(0, c, 29):
                ref = fp4.attend(q[row + i], kc[o:o + e], vc[o:o + e], np.arange(e - c + i + 1))
                err = np.abs(out[row + i].double().cpu().numpy() - ref)
                # bf16 output (2^-8) and bf16 weights, whose error is at most 2^-8 of the mean magnitude
                assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * np.abs(vc[o:o + e]).max()).all(), (b, i, err.max())
            row += c
    st.batch.seq_lens.copy_(i32(done))
    st.build_block_sums()
    for _ in range(steps):
        done = [e + 1 for e in done]
        t.seq_lens.copy_(i32(done))
        t.q_len.copy_(i32(done))
        for x in (*st.k_new, *st.v_new, *t.q):
            x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
        st.k_idx_new.copy_(torch.stack([t.k_idx[o + e - 1:o + e] for o, e in zip(offs, done)]))
        st.step()
        torch.cuda.synchronize()
        _check(st)
        _check_new_rows(st)
    for b, o in enumerate(offs):  # the prompts' rows are still in the cache
        k, v = _cache(st, 0, b)
        n = first[b] + second[b]
        assert np.array_equal(k[:n], kc[o:o + n]) and np.array_equal(v[:n], vc[o:o + n])
