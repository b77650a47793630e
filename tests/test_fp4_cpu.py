"""The 4-bit cache without a GPU: its definitions against torch's own types, and the refusals of lsa_store_fp4 and
lsa_attend_fp4 before any launch."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import bench
import fp4_plain as fp4
from long_context_sparse_lsa_b200 import binding as lsa
from long_context_sparse_lsa_b200 import workloads as wls
from long_context_sparse_lsa_b200 import build
from long_context_sparse_lsa_b200.pipeline import LsaStep

P = 0x10000  # a fake, aligned device address: never dereferenced (the call is refused first)


def test_e4m3_table_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, fp4.E4M3)


def test_rounding_ties_to_even_code():
    assert fp4.nearest(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), fp4.E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6]
    x = np.abs(np.random.default_rng(0).normal(size=4096)) * np.exp2(np.random.default_rng(1).integers(-12, 10, 4096))
    want = torch.tensor(np.minimum(x, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    # (float first: none of these draws lies within a float's rounding of a tie)
    assert np.array_equal(fp4.nearest(np.minimum(x, 448), fp4.E4M3), want)


def test_quantise_small_examples():
    x = torch.zeros(128, dtype=torch.bfloat16)
    x[:16] = torch.tensor([6, -6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, 0.5, -0.5, 4, 3, 2, 1.5])
    codes, groups, vals = fp4.quantise(x, 1.0)
    assert groups.tolist() == [0x38] + [0] * 7  # 1.0, then empty groups
    assert vals[:16].tolist() == [6, -6, 4, 4, 2, 2, 1, 1, 0, 0, 0.5, -0.5, 4, 3, 2, 1.5]
    assert codes[0] == 0x7 | 0xF << 4 and codes[4] == 0x0 | 0x8 << 4


# ---- refusals --------------------------------------------------------------------------------------------------------


def _prompts(**kw):
    f = dict(n_seq=2, n_rows=8, max_len=100, reserved=0, total_tokens=100, row_offset=P, kv_offset=P, seq_lens=P)
    f.update(kw)
    return lsa._Prompts(*[f[n] for n, _ in lsa._Prompts._fields_])


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def _ptrs(*xs):
    return ctypes.addressof(_ptrs.keep.setdefault(xs, (ctypes.c_void_p * len(xs))(*xs)))


_ptrs.keep = {}


def _scales(*xs):
    return ctypes.addressof(_scales.keep.setdefault(xs, (ctypes.c_float * len(xs))(*xs)))


_scales.keep = {}


def _store(**kw):
    two = _ptrs(P, P)
    a = dict(kn=two, ks=512, vn=two, vs=512, H=4, d=128, prompts=_prompts(), layers=2, ksc=_scales(1.0, 0.5),
             vsc=_scales(1.0, 2.0 ** -100), k=two, kg=two, v=two, vg=two, kr=None, vr=None)
    a.update(kw)
    return lsa.load_library().lsa_store_fp4(a["kn"], a["ks"], a["vn"], a["vs"], a["H"], a["d"], _ref(a["prompts"]), a["layers"],
                                            a["ksc"], a["vsc"], a["k"], a["kg"], a["v"], a["vg"], a["kr"], a["vr"], None,
                                            None)


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.mark.parametrize("kw,want", [
    (dict(kn=None), INVALID), (dict(v=None), INVALID), (dict(kg=None), INVALID), (dict(ksc=None), INVALID),
    (dict(H=0), INVALID), (dict(H=257, ks=1 << 20, vs=1 << 20), UNSUPPORTED), (dict(d=64), UNSUPPORTED),
    (dict(layers=0), INVALID), (dict(layers=9), UNSUPPORTED),
    (dict(ks=504), INVALID), (dict(ks=516), INVALID), (dict(vs=0), INVALID),
    (dict(kr=_ptrs(P, P)), INVALID),  # one of the two rounded outputs
    (dict(kr=_ptrs(P, P + 8), vr=_ptrs(P, P)), INVALID),
    (dict(ksc=_scales(1.0, 0.75)), INVALID), (dict(ksc=_scales(1.0, 0.0)), INVALID),
    (dict(ksc=_scales(-1.0, 1.0)), INVALID), (dict(vsc=_scales(1.0, float("nan"))), INVALID),
    (dict(vsc=_scales(float("inf"), 1.0)), INVALID), (dict(vsc=_scales(2.0 ** -101, 1.0)), INVALID),
    (dict(k=_ptrs(P, P + 8)), INVALID), (dict(vg=_ptrs(P, P + 4)), INVALID), (dict(vn=_ptrs(P, None)), INVALID),
    (dict(prompts=None), INVALID), (dict(prompts=_prompts(n_seq=0)), INVALID),
    (dict(prompts=_prompts(n_rows=-1)), INVALID), (dict(prompts=_prompts(max_len=0)), INVALID),
    (dict(prompts=_prompts(reserved=1)), INVALID), (dict(prompts=_prompts(row_offset=None)), INVALID),
    (dict(prompts=_prompts(kv_offset=P + 4)), INVALID), (dict(prompts=_prompts(n_rows=1 << 30)), UNSUPPORTED),
    (dict(prompts=_prompts(n_rows=0)), 0),  # nothing to do, nothing launched
])
def test_store_refuses_before_launch(kw, want):
    assert _store(**kw) == want


def _attend(**kw):
    two = _ptrs(P, P)
    b = lsa._Batch(1, 4, 100, 0, 100, P, P, None, P, P)
    a = dict(q=two, k=two, kg=two, v=two, vg=two, ksc=_scales(1.0, 0.3), vsc=_scales(1.0, -2.0), H=8, K=2, d=128, sets=P,
             budget=3136, batch=b, G=2, out=two, ws=None, nb=0)
    a.update(kw)
    return lsa.load_library().lsa_attend_fp4(a["q"], a["k"], a["kg"], a["v"], a["vg"], a["ksc"], a["vsc"], a["H"], a["K"],
                                             a["d"], a["sets"], a["budget"], _ref(a["batch"]), a["G"], a["out"], a["ws"],
                                             a["nb"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(vg=None), INVALID), (dict(ksc=None), INVALID), (dict(out=None), INVALID),
    (dict(sets=None), INVALID), (dict(sets=P + 2), INVALID), (dict(budget=-1), INVALID), (dict(budget=16385), UNSUPPORTED),
    (dict(H=7), INVALID), (dict(H=6), UNSUPPORTED), (dict(H=64), UNSUPPORTED), (dict(d=64), UNSUPPORTED),
    (dict(G=0), INVALID), (dict(G=9), UNSUPPORTED), (dict(ksc=_scales(1.0, float("inf"))), INVALID),
    (dict(kg=_ptrs(P, P + 2)), INVALID), (dict(out=_ptrs(P, None)), INVALID), (dict(batch=None), INVALID),
    (dict(batch=lsa._Batch(1, 70000, 100, 0, 100, P, P, None, P, P)), UNSUPPORTED),
    (dict(batch=lsa._Batch(1, 0, 100, 0, 100, P, P, None, P, P)), 0),
    (dict(ws=None, nb=1 << 30), WORKSPACE), (dict(ws=P, nb=1), WORKSPACE), (dict(ws=P + 16, nb=1 << 30), WORKSPACE),
])
def test_attend_refuses_before_launch(kw, want):
    assert _attend(**kw) == want


def test_attend_workspace_follows_the_splits():
    size = lambda n_q, budget: lsa.load_library().lsa_attend_fp4_workspace_size(
        lsa._Batch(1, n_q, 100, 0, 100, P, P, None, P, P), 32, 4, 128, budget, 1)
    launches = lambda n_q, budget: lsa.load_library().lsa_attend_fp4_launches(
        lsa._Batch(1, n_q, 100, 0, 100, P, P, None, P, P), 32, 4, 128, budget, 1)
    assert size(4, 0) == 0 and launches(4, 0) == 1         # nothing selected: one split
    assert size(1000, 3136) == 0 and launches(1000, 3136) == 1  # more rows than SMs
    assert size(1, 3136) > 0 and launches(1, 3136) == 2
    assert size(0, 3136) == 0 and launches(0, 3136) == 0


def test_binding_refuses_wrong_tensors():
    t = lambda dtype, *s: torch.zeros(s, dtype=dtype)
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    pr = lsa.Prompts(t(torch.int32, 2), t(torch.int64, 1), t(torch.int32, 1), 3, 10, 10)
    ok = dict(k_new=[t(bf, 3, 2, 128)], v_new=[t(bf, 3, 2, 128)], k=[t(u8, 10, 2, 64)], k_group=[t(u8, 10, 2, 8)],
              v=[t(u8, 10, 2, 64)], v_group=[t(u8, 10, 2, 8)], k_scale=[1.0], v_scale=[1.0], prompts=pr)
    for kw, err in [(dict(k_new=[t(f32, 3, 2, 128)]), TypeError), (dict(v_new=[]), ValueError),
                    (dict(v_new=[t(bf, 4, 2, 128)]), TypeError), (dict(k=[t(u8, 10, 2, 128)]), TypeError),
                    (dict(v_group=[t(u8, 8, 2, 10).permute(2, 1, 0)]), TypeError), (dict(k_scale=[]), ValueError),
                    (dict(k_new=[t(bf, 3, 128, 2).transpose(1, 2)]), ValueError),
                    (dict(k_round=[t(bf, 3, 2, 128)]), ValueError),
                    (dict(prompts=lsa.Prompts(pr.row_offset, pr.kv_offset, pr.seq_lens, 4, 10, 10)), ValueError),
                    (dict(prompts=lsa.Prompts(pr.row_offset, pr.kv_offset, pr.seq_lens, 3, 10, 11)), ValueError),
                    (dict(prompts=lsa.Prompts(pr.row_offset.long(), pr.kv_offset, pr.seq_lens, 3, 10, 10)), TypeError),
                    (dict(prompts=lsa.Prompts(pr.row_offset[:1], pr.kv_offset, pr.seq_lens, 3, 10, 10)), ValueError),
                    (dict(dev_status=t(u8, 1)), TypeError), (dict(), ValueError)]:  # (the last: host tensors)
        with pytest.raises(err):
            lsa.lsa_store_fp4(**{**ok, **kw}, stream=0)
    b = lsa.Batch(t(torch.int64, 1), t(torch.int32, 1), t(torch.int32, 3), t(torch.int32, 3), 10, 10)
    ok = dict(q=[t(bf, 3, 8, 128)], k=[t(u8, 10, 2, 64)], k_group=[t(u8, 10, 2, 8)], v=[t(u8, 10, 2, 64)],
              v_group=[t(u8, 10, 2, 8)], k_scale=[1.0], v_scale=[1.0], index_sets=t(torch.int32, 3, 16), batch=b,
              out=[t(f32, 3, 8, 128)], workspace=None)
    for kw, err in [(dict(q=[t(f32, 3, 8, 128)]), TypeError), (dict(out=[t(bf, 3, 8, 128)]), TypeError),
                    (dict(index_sets=t(torch.int64, 3, 16)), TypeError), (dict(index_sets=t(torch.int32, 2, 16)), TypeError),
                    (dict(k=[t(u8, 9, 2, 64)]), ValueError), (dict(v=[t(u8, 10, 1, 64)]), TypeError),
                    (dict(v_scale=[1.0, 1.0]), ValueError), (dict(q=[t(bf, 2, 8, 128)]), TypeError),
                    (dict(dev_status=t(u8, 1)), TypeError), (dict(), ValueError)]:
        with pytest.raises(err):
            lsa.lsa_attend_fp4(**{**ok, **kw}, stream=0)


def test_step_bytes_with_a_4_bit_cache():
    b16, b4 = bench.step_bytes(wls.BATCH128K), bench.step_bytes(wls.BATCH128K, kv_fp4=True)
    # per row and layer 3136 entries, K and V of 4 kv heads: 256 B there, 64 of codes and 8 of scales here
    assert b16["attend"] - b4["attend"] == 16 * 2 * 3136 * 4 * (256 - 72)
    # per sequence: the new token's K and V read as bf16 in both, written in 4 bits
    assert b16["append"] - b4["append"] == 16 * 2 * 4 * (256 - 72)
    assert b4["index"] == b16["index"]


def _step(wl, **kw):
    return LsaStep(wl, wls.make(wl, "cpu", with_kv=False), "cpu", kv_fp4=True, **kw)


def test_decode_step_over_a_4_bit_cache():
    """The step's buffers, launches and refusals, without a GPU."""
    small = wls.small(wls.BATCH128K, lens=(300, 70), drafts=2, G=2, seed=7)
    st = _step(small)
    assert st.k4[1].shape == (370, 4, 64) and st.v4_group[0].shape == (370, 4, 8)
    assert all(fp4.E4M3[0x20] == 0.125 <= fp4.E4M3[x.numpy()].min() and fp4.E4M3[x.numpy()].max() <= 0.9375
               for x in st.k4_group + st.v4_group)
    assert st.newest.row_offset.tolist() == [0, 2, 4] and st.k_new[1].shape == (2, 2, 4, 128)
    before = [x.clone() for x in [*st.k_new, *st.v_new]]
    st.pack_io()
    assert all(torch.equal(x, y) for x, y in zip(before, [*st.k_new, *st.v_new]))
    for wl in (wls.BATCH128K, wls.CTX1M):  # the store is a launch of its own
        cut = wls.small(wl, lens=tuple(min(n, 4096) for n in wl.lens))
        st, t = _step(cut), wls.make(cut, "cpu")
        st16 = LsaStep(cut, t, "cpu")
        for x in (st, st16):
            x.batch.max_len = max(wl.lens)
        assert st.kernels_per_step() == st16.kernels_per_step() + 1
    for kw in (dict(kv_fp8=True), dict(grouped=True), dict(si_attend=True)):
        with pytest.raises(ValueError):
            _step(small, **kw)
    chunk = _step(wls.small(wls.PREFILL, lens=(300,), prefill_new=20))
    assert chunk.n_new == 0 and not chunk.si_attend


@pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                    reason="nvcc not available")
def test_no_register_spills():
    """The kernels keep their fragments in registers; the 4-bit attention spills up to 36 bytes of addresses, outside
    its loop over the entries."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    for src, allowed in (("store_fp4.cu", 0), ("attend_fp4.cu", 36), ("attend_prompt.cu", 0), ("attend_prompt_few.cu", 0)):
        r = subprocess.run([nvcc, *build.ARCH, *build.NVCC_FLAGS, "-Xptxas", "-v", "-c", os.path.join(build.CSRC, src), "-o",
                            os.path.join(build.BUILD_DIR, "ptxas_check_fp4.o")], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        found = re.findall(r"Function properties for (\S+)\s+\d+ bytes stack frame, (\d+) bytes spill stores", r.stderr)
        assert found
        for fn, spill in found:
            assert int(spill) <= allowed, (fn, spill)
