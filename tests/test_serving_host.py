"""The serving operators' boundary without a GPU: struct layouts against the C
compiler, and every refusal of the host checks."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, NULL, ODD = ctypes.c_void_p(1 << 16), None, ctypes.c_void_p((1 << 16) + 4)
ARG, SHAPE, SCALE = 1, 2, 4


@pytest.fixture(scope="module")
def trit():
    from bit_plane_select_gb300 import build
    build.build()
    import bit_plane_select_gb300 as t
    return t


def structs(trit):
    return {"trit_kv_cache": trit.TritKvCache, "trit_kv_batch": trit.TritKvBatch,
            "trit_kv_append_job": trit.TritKvAppendJob, "trit_attn_job": trit.TritAttnJob,
            "trit_verify_job": trit.TritVerifyJob}


def test_struct_layouts_match_the_c_compiler(trit, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "trit.h"', "int main(void) {"]
    for c, cls in structs(trit).items():
        lines.append(f'printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in out.splitlines()}
    for c, cls in structs(trit).items():
        assert got[(c, "size")] == ctypes.sizeof(cls), c
        for f, _ in cls._fields_:
            assert got[(c, f)] == getattr(cls, f).offset, (c, f)


def cache(trit, **kw):
    a = dict(k=P, v=P, page_stride=5 * 64 * 128, head_stride=64 * 128, slot_stride=128, pages=10, heads=5,
             page_size=64, head_dim=128, dtype=1, reserved=0)
    a.update(kw)
    return trit.TritKvCache(**a)


def batch(trit, **kw):
    a = dict(prefix_table=P, table=P, lens=P, new_lens=NULL, prefix_len=100, table_stride=8, prefix_pages=2,
             table_pages=8, B=3, T=2)
    a.update(kw)
    return trit.TritKvBatch(**a)


BAD_CACHE = [(dict(k=NULL), ARG), (dict(v=NULL), ARG), (dict(k=ODD), ARG), (dict(slot_stride=130), ARG),
             (dict(page_stride=-8), ARG), (dict(dtype=0), ARG), (dict(dtype=3), ARG), (dict(reserved=1), ARG),
             (dict(head_dim=96), SHAPE), (dict(pages=0), SHAPE), (dict(heads=0), SHAPE), (dict(page_size=0), SHAPE)]
BAD_BATCH = [(dict(table=NULL), ARG), (dict(lens=NULL), ARG), (dict(prefix_table=NULL), ARG), (dict(B=0), SHAPE),
             (dict(B=4097), SHAPE), (dict(T=0), SHAPE), (dict(table_pages=0), SHAPE), (dict(table_stride=7), SHAPE),
             (dict(prefix_len=129), SHAPE), (dict(prefix_len=-1), SHAPE), (dict(prefix_pages=-1), SHAPE)]


def append_job(trit, c=None, b=None, **kw):
    a = dict(cache=c or cache(trit), batch=b or batch(trit), q=P, k=P, v=P, q_out=P, cos=P, sin=P, q_gain=NULL,
             k_gain=NULL, q_stride=2560, k_stride=640, v_stride=640, max_pos=1000, eps=1e-5, q_heads=20, rot=128,
             src_dtype=0, flags=0, reserved=0)
    a.update(kw)
    return trit.TritKvAppendJob(**a)


def test_append_refusals(trit):
    fn = trit.lib().trit_kv_append
    for kw, code in BAD_CACHE:
        assert fn(ctypes.byref(append_job(trit, c=cache(trit, **kw))), P, NULL) == code, kw
    for kw, code in BAD_BATCH:
        assert fn(ctypes.byref(append_job(trit, b=batch(trit, **kw))), P, NULL) == code, kw
    for kw, code in [(dict(k=NULL), ARG), (dict(v=NULL), ARG), (dict(q=NULL), ARG), (dict(q_out=NULL), ARG),
                     (dict(cos=NULL), ARG), (dict(k=ODD), ARG), (dict(q_gain=ODD), ARG), (dict(flags=2), ARG),
                     (dict(reserved=1), ARG), (dict(src_dtype=2), ARG), (dict(q_stride=2561), ARG),
                     (dict(v_stride=-640), ARG), (dict(rot=136), SHAPE), (dict(rot=4), SHAPE), (dict(rot=-8), SHAPE),
                     (dict(max_pos=-1), SHAPE), (dict(q_heads=21), SHAPE), (dict(q_heads=0), SHAPE),
                     (dict(q_gain=P, eps=-1.0), SCALE), (dict(k_gain=P, eps=float("nan")), SCALE)]:
        assert fn(ctypes.byref(append_job(trit, **kw)), P, NULL) == code, kw
    assert fn(ctypes.byref(append_job(trit, b=batch(trit, B=4096, T=1 << 20))), P, NULL) == SHAPE
    assert fn(ctypes.byref(append_job(trit)), NULL, NULL) == ARG
    assert fn(None, P, NULL) == ARG


def test_attn_refusals(trit):
    L = trit.lib()

    def job(c=None, b=None, **kw):
        a = dict(cache=c or cache(trit), batch=b or batch(trit), q=P, out=P, lse=NULL, workspace=P,
                 workspace_bytes=1 << 40, q_stride=2560, scale=0.1, q_heads=20, out_dtype=0, flags=0)
        a.update(kw)
        return trit.TritAttnJob(**a)
    fn = L.trit_attn_paged
    assert L.trit_attn_workspace_bytes(ctypes.byref(job())) > 0
    for kw, code in BAD_CACHE:
        assert fn(ctypes.byref(job(c=cache(trit, **kw))), P, NULL) == code, kw
        assert L.trit_attn_workspace_bytes(ctypes.byref(job(c=cache(trit, **kw)))) == -1
    for kw, code in BAD_BATCH:
        assert fn(ctypes.byref(job(b=batch(trit, **kw))), P, NULL) == code, kw
    need = L.trit_attn_workspace_bytes(ctypes.byref(job()))
    for kw, code in [(dict(q=NULL), ARG), (dict(out=NULL), ARG), (dict(workspace=NULL), ARG), (dict(q=ODD), ARG),
                     (dict(out=ODD), ARG), (dict(lse=ctypes.c_void_p(65538)), ARG), (dict(q_stride=2564), ARG),
                     (dict(q_stride=-8), ARG), (dict(flags=1), ARG), (dict(out_dtype=2), ARG),
                     (dict(q_heads=21), SHAPE), (dict(q_heads=0), SHAPE), (dict(scale=float("inf")), SCALE),
                     (dict(workspace_bytes=need - 1), 8)]:
        assert fn(ctypes.byref(job(**kw)), P, NULL) == code, kw
    assert fn(ctypes.byref(job(b=batch(trit, B=4096, T=1 << 20))), P, NULL) == SHAPE
    assert fn(ctypes.byref(job()), NULL, NULL) == ARG
    assert fn(None, P, NULL) == ARG
    assert L.trit_attn_workspace_bytes(None) == -1


def test_verify_refusals(trit):
    fn = trit.lib().trit_draft_verify

    def job(**kw):
        a = dict(p=P, q=P, draft=P, n_draft=NULL, u=P, race=P, tokens=P, accepted=P,
                 p_seq_stride=500, p_tok_stride=100, q_seq_stride=400, q_tok_stride=100, race_stride=100, V=100,
                 B=2, T=4, dtype=0, flags=0)
        a.update(kw)
        return trit.TritVerifyJob(**a)
    half = ctypes.c_void_p((1 << 16) + 2)
    for kw, code in [(dict(p=NULL), ARG), (dict(q=NULL), ARG), (dict(draft=NULL), ARG), (dict(u=NULL), ARG),
                     (dict(race=NULL), ARG), (dict(tokens=NULL), ARG), (dict(accepted=NULL), ARG),
                     (dict(accepted=NULL), ARG), (dict(p=half), ARG),
                     (dict(dtype=3), ARG), (dict(flags=1), ARG), (dict(p_tok_stride=-1), ARG), (dict(V=0), SHAPE),
                     (dict(B=0), SHAPE), (dict(B=65536), SHAPE), (dict(T=0), SHAPE), (dict(V=1 << 31), SHAPE)]:
        assert fn(ctypes.byref(job(**kw)), P, NULL) == code, kw
    assert fn(ctypes.byref(job()), NULL, NULL) == ARG
    assert fn(None, P, NULL) == ARG


def test_python_checks(trit):
    """CPU tensors, wrong types and shapes raise before anything is called."""
    torch = pytest.importorskip("torch")
    cpu = torch.zeros(2, 5, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        trit.KvCache(cpu, cpu)
    with pytest.raises(ValueError, match="strides"):
        trit.KvCache(cpu, cpu.transpose(1, 2))
    with pytest.raises(ValueError, match="prefix_table"):
        trit.KvBatch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1, prefix_len=3)
    with pytest.raises(ValueError, match="CUDA"):
        trit.Rope(torch.zeros(4, 4), torch.zeros(4, 4))
