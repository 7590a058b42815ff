"""Host-side checks of the paged latent cache's calls: every refusal comes back before any launch (no GPU here)."""
import ctypes
import os
import subprocess

import pytest
import torch

from mla_latent_kv_31_b200 import build as mla_build
from mla_latent_kv_31_b200 import mla, synth
from paged_testlib import Case, rope

OK, INVALID, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
P = 1 << 20                                             # an aligned address that no call reads


@pytest.fixture(scope="module", autouse=True)
def built():
    mla_build.build()


def batch(**over):
    b = mla.MlaPaged(P, 100, 64, P, 20, 20, P, P, 4, 8)
    for k, v in over.items():
        setattr(b, k, v)
    return ctypes.byref(b)


def calls(h, b):
    """The status of each paged call with this batch and otherwise sound arguments (too small a workspace where
    the call takes one, so that a sound batch ends there)."""
    L = mla.lib()
    return {"append": lambda: L.mla_paged_append(h, b, P, 576, P, P, P, None),
            "attn": lambda: L.mla_attn_paged(h, b, P, P, P, P, None, 0, None),
            "sparse": lambda: L.mla_attn_paged_sparse(h, b, P, P, P, 4, P, P, None, 0, None),
            "select": lambda: L.mla_paged_select(h, b, P, P, P, 8, 1, 1, P, P, 0, None)}


@pytest.mark.parametrize("over", [dict(cache=None), dict(block_table=None), dict(cu_q=None), dict(kv_lens=None),
                                  dict(B=0), dict(total_q=0), dict(num_pages=0), dict(max_pages=0),
                                  dict(table_stride=19), dict(page_size=0), dict(page_size=-16), dict(page_size=24),
                                  dict(page_size=8), dict(num_pages=1 << 31), dict(num_pages=(1 << 31) // 64),
                                  dict(total_q=1 << 40), dict(B=1 << 30),
                                  dict(max_pages=(1 << 24) + 1, table_stride=1 << 25)])    # more than 2^30 rows
def test_bad_batches_are_refused(over):
    h = mla.mla_create(synth.V3)
    try:
        for name, call in calls(h, batch(**over)).items():
            assert call() == INVALID, name
    finally:
        mla.mla_destroy(h)


def test_misaligned_pointers_are_refused():
    h = mla.mla_create(synth.V3)
    try:
        for field in ("cache", "block_table", "cu_q", "kv_lens"):
            for name, call in calls(h, batch(**{field: P + 8})).items():
                assert call() == ALIGN, (field, name)
        L, b = mla.lib(), batch()
        assert L.mla_paged_append(h, b, P + 2, 576, None, None, None, None) == ALIGN
        assert L.mla_paged_append(h, b, P, 576, P + 4, P, None, None) == ALIGN
        assert L.mla_paged_append(h, b, P, 576, None, None, P + 8, None) == ALIGN
        assert L.mla_attn_paged(h, b, P, P + 2, P, P, None, 0, None) == ALIGN
        assert L.mla_attn_paged_sparse(h, b, P, P, P + 4, 4, P, P, None, 0, None) == ALIGN
        assert L.mla_paged_select(h, b, P, P, P, 8, 1, 1, P + 4, P, 0, None) == ALIGN
    finally:
        mla.mla_destroy(h)


def test_arguments_of_each_call():
    h = mla.mla_create(synth.V3)
    L, b = mla.lib(), batch()
    try:
        assert L.mla_paged_append(None, b, P, 576, None, None, None, None) == INVALID
        assert L.mla_paged_append(h, None, P, 576, None, None, None, None) == INVALID
        assert L.mla_paged_append(h, b, None, 576, None, None, None, None) == INVALID
        assert L.mla_paged_append(h, b, P, 568, None, None, None, None) == INVALID      # rows overlap
        assert L.mla_paged_append(h, b, P, 580, None, None, None, None) == INVALID      # not 16-byte rows
        assert L.mla_paged_append(h, b, P, 576, P, None, None, None) == INVALID         # q_rope without q_out
        assert L.mla_attn_paged(h, b, P, P, None, P, None, 0, None) == INVALID
        assert L.mla_attn_paged_sparse(h, b, P, P, None, 4, P, P, None, 0, None) == INVALID
        for top_k in (0, -1, -(1 << 31), 1 << 21):
            assert L.mla_attn_paged_sparse(h, b, P, P, P, top_k, P, P, None, 0, None) == INVALID
            assert L.mla_paged_select(h, b, P, P, P, top_k, 0, 1, P, P, 1 << 40, None) == INVALID
        for first, last in ((-1, 1), (0, 0), (4, 5), (1 << 30, 1 << 30)):
            assert L.mla_paged_select(h, b, P, P, P, 8, first, last, P, P, 1 << 40, None) == INVALID
        assert L.mla_paged_select(h, batch(total_q=70000), P, P, P, 8, 1, 1, P, P, 1 << 40, None) == INVALID
        assert L.mla_paged_select(h, b, P, P, None, 8, 1, 1, P, P, 1 << 40, None) == INVALID
        assert L.mla_paged_select(h, b, P, P, P, 8, 1, 1, P, P, 0, None) == WORKSPACE
        mla.mla_set_cache_format(h, mla.CACHE_FP8)
        for name, call in calls(h, b).items():
            assert call() == UNSUPPORTED, name
    finally:
        mla.mla_destroy(h)


@pytest.mark.parametrize("device", [0, 1, "cuda:1", torch.device("cuda", 0), torch.device("cuda"), None])
def test_default_stream_takes_every_name_of_a_device(monkeypatch, device):
    """Without a stream, a call goes to torch's current stream of the device, named as torch.cuda names devices."""
    class Stream:
        cuda_stream = 77
    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: asked.append(d) or Stream)
    assert mla._stream(None, device) == 77 and asked == [device]
    assert mla._stream(5, device) == 5 and mla._stream(Stream, device) == 77 and asked == [device]


def test_workspaces_and_summary_rows():
    h = mla.mla_create(synth.V3)
    t = mla.mla_create(synth.TINY, mla.MLA_FP32)
    odd = mla.mla_create(synth.Dims(d=8, n_h=1, d_h=4, d_c=7, d_cq=4, d_r=2), mla.MLA_FP32)
    try:
        assert mla.mla_paged_summary_bytes(h) == 592 and mla.mla_paged_summary_bytes(t) == 96
        with pytest.raises(mla.MLAError) as e:
            mla.mla_paged_summary_bytes(odd)            # 9 codes do not end on a multiple of 4
        assert e.value.status == UNSUPPORTED
        assert mla.lib().mla_paged_append(odd, batch(), P, 9, None, None, P, None) == UNSUPPORTED
        for f in (mla.mla_attn_paged_workspace, mla.mla_paged_select_workspace):
            for x, y in ((0, 1), (1, 0), (-1, 1)):
                with pytest.raises(mla.MLAError):
                    f(h, x, y)
        n, r = synth.V3.n_h, 2 ** 31 - 1
        assert mla.mla_attn_paged_workspace(h, 1 << 20, r // n) > r // n * 16
        assert mla.mla_paged_select_workspace(h, 65535, 1 << 26) > 65535 << 28
        for f, x, y in ((mla.mla_attn_paged_workspace, 1, r // n + 1), (mla.mla_attn_paged_workspace, (1 << 20) + 1, 1),
                        (mla.mla_attn_paged_workspace, 1, 1 << 60), (mla.mla_paged_select_workspace, 65536, 1),
                        (mla.mla_paged_select_workspace, 1, (1 << 26) + 1), (mla.mla_paged_select_workspace, 1 << 62, 1 << 62)):
            with pytest.raises(mla.MLAError) as e:      # sizes that no call takes: their bytes would wrap around
                f(h, x, y)
            assert e.value.status == INVALID
        small, large = (mla.mla_paged_select_workspace(h, 4, n) for n in (10, 2000))
        assert 4 * 2000 * 4 <= large and small < large
    finally:
        for x in (h, t, odd):
            mla.mla_destroy(x)


def test_binding_checks_shapes_types_and_strides():
    c = Case("fp32", 16, [20, 40], [1, 3], device="cpu")
    mla.PagedBatch(c.cache, c.table, c.cu, c.d_lens, 4)
    mla.PagedBatch(c.cache, c.table[:, :2], c.cu, c.d_lens, 4)          # a slice of a wider table
    for bad in ((c.cache, c.table.long(), c.cu, c.d_lens), (c.cache, c.table, c.cu.int(), c.d_lens),
                (c.cache, c.table, c.cu[:-1], c.d_lens), (c.cache, c.table[:1], c.cu, c.d_lens),
                (c.cache[0], c.table, c.cu, c.d_lens), (c.cache, c.table[:, ::2], c.cu, c.d_lens),
                (c.cache[:, ::2], c.table, c.cu, c.d_lens)):
        with pytest.raises(ValueError):
            mla.PagedBatch(*bad, 4)
    m = mla.MLA(synth.TINY, None, mla.MLA_FP32)
    with pytest.raises(ValueError):                                      # a CPU cache
        m.attn_paged(mla.PagedBatch(c.cache, c.table, c.cu, c.d_lens, 4), c.q[..., :64].float(), c.q[..., 64:].float())
    m.close()


def test_the_tests_own_rotation_and_selection():
    """The plain forms that the GPU tests go by, against hand-made values."""
    d = synth.TINY
    x = torch.zeros(d.d_r, dtype=torch.float64)
    x[2] = 1.0
    y = rope(x, 5, d)
    a = 5 * d.rope_base ** (-2.0 / d.d_r)
    assert torch.allclose(y[2:4], torch.tensor([a, a], dtype=torch.float64).cos() * torch.tensor([1.0, 0.0])
                          + torch.tensor([a, a], dtype=torch.float64).sin() * torch.tensor([0.0, 1.0]))
    c = Case("fp32", 16, [16 * 9], [1], device="cpu")
    means = torch.zeros(c.num_pages, c.W, dtype=torch.float64)
    means[c.table[0, 5].long()] = c.q[0, 2]             # one block looks like a query, the others score 0
    assert c.select(means, 4, 1, 1)[0].tolist() == [0, 1, 5, 8]


def test_first_call_of_a_handle(tmp_path):
    """tests/handle_init.cu: threads that are first at once, and each runtime call failing, over a stand-in runtime."""
    exe = tmp_path / "handle_init"
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([mla_build.nvcc(), *mla_build.ARCH, *mla_build.FLAGS, "-cudart", "none",
                    os.path.join(here, "handle_init.cu"), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)
