"""lsa_attend_prompt without a GPU: its refusals before any launch, its workspace and the binding's checks."""
import pytest
import torch

from long_context_sparse_lsa_b200 import binding as lsa
from test_fp4_cpu import INVALID, P, UNSUPPORTED, WORKSPACE, _prompts, _ref


def _prompt(**kw):
    a = dict(q=P, qs=4096, k=P, ks=512, v=P, vs=512, H=32, K=4, d=128, prompts=_prompts(n_rows=8000, max_len=9000), out=P,
             lse=P, ws=None, nb=0)
    a.update(kw)
    return lsa.load_library().lsa_attend_prompt(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["H"], a["K"], a["d"],
                                                _ref(a["prompts"]), a["out"], a["lse"], a["ws"], a["nb"], None, None)


few = dict(prompts=_prompts(n_seq=1, n_rows=1, max_len=9000))  # one row over a long cache: the keys are split


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(q=P + 8), INVALID), (dict(out=P + 16), INVALID), (dict(lse=P + 2), INVALID),
    (dict(qs=4088), INVALID), (dict(ks=516), INVALID), (dict(vs=0), INVALID), (dict(ks=1 << 40), UNSUPPORTED),
    (dict(H=0), INVALID), (dict(K=0), INVALID), (dict(H=30), INVALID), (dict(d=0), INVALID), (dict(d=64), UNSUPPORTED),
    (dict(H=260, qs=1 << 16), UNSUPPORTED), (dict(H=8192, K=1024, qs=1 << 20, ks=1 << 18, vs=1 << 18), UNSUPPORTED),
    (dict(prompts=None), INVALID), (dict(prompts=_prompts(n_seq=0)), INVALID), (dict(prompts=_prompts(reserved=2)), INVALID),
    (dict(prompts=_prompts(seq_lens=None)), INVALID), (dict(prompts=_prompts(total_tokens=0)), INVALID),
    (dict(prompts=_prompts(total_tokens=(1 << 31))), UNSUPPORTED), (dict(prompts=_prompts(n_rows=1 << 30)), UNSUPPORTED),
    (dict(prompts=_prompts(n_rows=0)), 0),
    (few, WORKSPACE), ({**few, "ws": P, "nb": 1}, WORKSPACE), ({**few, "ws": P + 16, "nb": 1 << 30}, WORKSPACE),
])
def test_refuses_before_launch(kw, want):
    assert _prompt(**kw) == want


def test_workspace_and_launches_follow_the_splits():
    lib = lsa.load_library()
    for n_seq, n_rows, max_len, split in [(1, 1, 9000, True), (1, 8000, 9000, False), (16, 16, 3136, True), (64, 64, 9000, True),
                                          (1, 1, 100, False), (4, 40, 9000, True),
                                          (16, 16, 1000, False), (4, 4, 2000, False), (9, 9, 2000, True)]:  # joined in clusters
        p = _prompts(n_seq=n_seq, n_rows=n_rows, max_len=max_len)
        assert lib.lsa_attend_prompt_launches(p, 32, 4, 128) == (2 if split else 1)
        assert (lib.lsa_attend_prompt_workspace_size(p, 32, 4, 128) > 0) == split
    assert lib.lsa_attend_prompt_workspace_size(_prompts(n_rows=0), 32, 4, 128) == 0
    assert lib.lsa_attend_prompt_launches(_prompts(), 32, 5, 128) == 0


def test_binding_refuses_wrong_tensors():
    t = lambda dtype, *s: torch.zeros(s, dtype=dtype)
    bf = torch.bfloat16
    pr = lsa.Prompts(t(torch.int32, 2), t(torch.int64, 1), t(torch.int32, 1), 3, 10, 10)
    ok = dict(q=t(bf, 3, 8, 128), k=t(bf, 10, 2, 128), v=t(bf, 10, 2, 128), prompts=pr, out=t(bf, 3, 8, 128))
    for kw, err in [(dict(q=t(torch.float16, 3, 8, 128)), TypeError), (dict(out=t(torch.float32, 3, 8, 128)), TypeError),
                    (dict(v=t(bf, 10, 1, 128)), ValueError), (dict(v=t(bf, 9, 2, 128)), ValueError),
                    (dict(k=t(bf, 9, 2, 128), v=t(bf, 9, 2, 128)), ValueError), (dict(out=t(bf, 3, 4, 128)), ValueError),
                    (dict(out=t(bf, 3, 16, 128)[:, ::2]), ValueError), (dict(q=t(bf, 3, 16, 128)[:, ::2]), ValueError),
                    (dict(q=t(bf, 2, 8, 128), out=t(bf, 2, 8, 128)), ValueError),
                    (dict(lse=t(bf, 3, 8)), TypeError), (dict(lse=t(torch.float32, 8, 3).T), TypeError),
                    (dict(dev_status=t(bf, 1)), TypeError), (dict(), ValueError)]:  # (the last: host tensors)
        with pytest.raises(err):
            lsa.lsa_attend_prompt(**{**ok, **kw}, stream=0)


def test_binding_refuses_an_expanded_workspace():
    """Its elements are more than the bytes behind its address."""
    t = lambda dtype, *s: torch.zeros(s, dtype=dtype)
    bf, u8 = torch.bfloat16, torch.uint8
    wide = t(u8, 1).expand(1 << 30)
    pr = lsa.Prompts(t(torch.int32, 2), t(torch.int64, 1), t(torch.int32, 1), 3, 10, 10)
    b = lsa.Batch(t(torch.int64, 1), t(torch.int32, 1), t(torch.int32, 3), t(torch.int32, 3), 10, 10)
    q, kv, sets, out = t(bf, 3, 8, 128), t(bf, 10, 2, 128), t(torch.int32, 3, 1024), t(torch.float32, 3, 8, 128)
    for ws in (wide, t(u8, 4096)[::2]):
        with pytest.raises(TypeError, match="workspace"):
            lsa.lsa_attend_prompt(q, kv, kv, pr, torch.empty_like(q), ws, stream=0)
        with pytest.raises(TypeError, match="workspace"):
            lsa.lsa_attend_fp4([q], [t(u8, 10, 2, 64)], [t(u8, 10, 2, 8)], [t(u8, 10, 2, 64)], [t(u8, 10, 2, 8)], [1.0], [1.0],
                               sets, b, [out], ws, stream=0)
    # the calls that take any tensor count what lies behind the address (refused before any launch)
    assert lsa._bytes(wide) == 1 and lsa._bytes(t(torch.float32, 6, 2).T) == 48 and lsa._bytes(t(u8, 0)) == 0
    assert lsa._bytes(None) == 0 and lsa._bytes(t(u8, 8)[::2]) == 4
    need = lsa.lsa_attend_workspace_size(b, 8, 2, 128, 1024, 1)
    assert need > 1
    for ws in (t(u8, 1).expand(need), None):
        with pytest.raises(lsa.LsaError) as e:
            lsa.lsa_attend([q], [kv], [kv], sets, b, [out], ws, stream=0)
        assert e.value.status == WORKSPACE


@pytest.mark.parametrize("n_seq,n_rows,H,K", [(1, 100, 32, 4), (1, 1, 32, 4), (3, 700, 8, 8), (200, 200, 16, 1)])
def test_the_plan_takes_any_bound_on_the_lengths(n_seq, n_rows, H, K):
    """The largest max_len, as a caller without a bound gives it, is planned like one a little below."""
    lib = lsa.load_library()
    plans = [(lib.lsa_attend_prompt_workspace_size(p, H, K, 128), lib.lsa_attend_prompt_launches(p, H, K, 128))
             for p in (_prompts(n_seq=n_seq, n_rows=n_rows, max_len=m) for m in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 300))]
    assert plans[0] == plans[1] == plans[2] and plans[0][1] == 2
