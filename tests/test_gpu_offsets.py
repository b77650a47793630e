"""Cache offsets so large that offset + length passes 2^63: the sequence is flagged and skipped like any that lies outside
the caches, by every call, and the other sequences are served as before."""
import pytest
import torch

from long_context_sparse_lsa_b200 import binding as lsa
from long_context_sparse_lsa_b200 import workloads as wls
from long_context_sparse_lsa_b200.pipeline import LsaStep

pytestmark = pytest.mark.gpu
DEV = "cuda"
FAR = 2 ** 63 - 1


def _step(hi, lens=(900, 700), drafts=1, **kw):
    wl = wls.small(wls.BATCH128K, name="far", lens=lens, drafts=drafts, hi_block=64 if hi else 0, hi_topblocks=4 if hi else 0, topk=200,
                   window=150, sink=16, G=2, seed=3)
    st = LsaStep(wl, wls.make(wl, DEV), DEV, **kw)
    st.build_block_sums()
    return st


@pytest.mark.parametrize("hi,name", [(False, "kv_offset"), (True, "kv_offset"), (True, "blk_offset")])
@pytest.mark.parametrize("far", [FAR, FAR - 100])
@pytest.mark.parametrize("kw", [{}, dict(kv_fp8=True), dict(kv_fp4=True), dict(grouped=True, drafts=2), dict(fuse_append=False)])
def test_decode_step(hi, name, far, kw):
    st = _step(hi, **kw)
    st.step()
    assert st.status_bits() == 0
    sets, out = st.sets.clone(), [x.clone() for x in st.out]
    getattr(st.t, name)[1] = far
    calls = [st.build_block_sums, st.append, st.index, st.step] + ([st.attend] if name == "kv_offset" else [])
    for call in calls:
        if call == st.build_block_sums and not hi:
            continue
        st.status.zero_()
        call()
        assert st.status_bits() & lsa.LSA_DEV_BAD_LENGTH, call
    n = st.wl.drafts  # the rows of sequence 0
    assert torch.equal(st.sets[:n], sets[:n]) and all(torch.equal(x[:n], y[:n]) for x, y in zip(st.out, out))


@pytest.mark.parametrize("hi", [False, True])
def test_prefill_chunk(hi):
    wl = wls.small(wls.PREFILL, name="far_chunk", lens=(1500,), prefill_new=40, hi_block=64 if hi else 0, hi_topblocks=4 if hi else 0,
                   topk=200, window=150, sink=16, G=1, seed=3)
    st = LsaStep(wl, wls.make(wl, DEV), DEV)
    st.build_block_sums()
    st.step()
    assert st.status_bits() == 0
    st.t.kv_offset[0] = FAR
    for call in (st.index, st.attend):
        st.status.zero_()
        call()
        assert st.status_bits() & lsa.LSA_DEV_BAD_LENGTH


@pytest.mark.parametrize("rows", [[1, 1, 1], [40, 30, 20], [300, 200, 100]])
@pytest.mark.parametrize("far", [FAR, FAR - 100])
def test_prompts_and_their_store(rows, far):
    lens = [600, 500, 400]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ro = [0, rows[0], rows[0] + rows[1], sum(rows)]
    ko = torch.tensor([0, 600, 1100], dtype=torch.int64, device=DEV)
    pr = lsa.Prompts(i32(ro), ko, i32(lens), ro[3], 600, 1500)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = rand(ro[3], 8, 128), rand(1500, 2, 128), rand(1500, 2, 128)
    ws = torch.empty(max(256, lsa.lsa_attend_prompt_workspace_size(pr, 8, 2, 128)), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def attend():
        out = torch.full_like(q, 9.0)
        lsa.lsa_attend_prompt(q, k, v, pr, out, ws, dev_status=status)
        return out

    def store():
        c = [torch.full((1500, 2, n), 0xA5, dtype=torch.uint8, device=DEV) for n in (64, 8, 64, 8)]
        lsa.lsa_store_fp4([k[:ro[3]]], [v[:ro[3]]], *[[x] for x in c], [1.0], [1.0], pr, dev_status=status)
        return c

    near, stored = attend(), store()
    assert status.item() == 0
    ko[1] = far
    got = attend()
    assert status.item() == lsa.LSA_DEV_BAD_LENGTH
    near[ro[1]:ro[2]] = 9.0
    assert torch.equal(got, near)
    status.zero_()
    got = store()
    assert status.item() == lsa.LSA_DEV_BAD_LENGTH
    for x, y in zip(got, stored):
        y[600:1100] = 0xA5
        assert torch.equal(x, y)
