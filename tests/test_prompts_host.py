"""The boundary of prompts, of the 4-bit cache and of scoring without a GPU: struct layouts
against the C compiler, and every refusal of the host checks."""
import ctypes
import os
import shutil
import subprocess

import pytest

from test_serving_host import ARG, BAD_BATCH, NULL, ODD, P, SCALE, SHAPE, batch, trit  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BYTE = ctypes.c_void_p((1 << 16) + 1)


def test_struct_layouts_match_the_c_compiler(trit, tmp_path):  # noqa: F811
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"trit_kv4_cache": trit.TritKv4Cache, "trit_kv4_append_job": trit.TritKv4AppendJob,
               "trit_kv4_read_job": trit.TritKv4ReadJob, "trit_attn4_job": trit.TritAttn4Job,
               "trit_prompt_job": trit.TritPromptJob, "trit_logprob_job": trit.TritLogprobJob}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "trit.h"', "int main(void) {"]
    for c, cls in structs.items():
        lines.append(f'printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in cls._fields_]
    lines.append('printf("group value %d\\nmost value %d\\n", TRIT_KV4_GROUP, TRIT_MAX_TOP);')
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in out.splitlines()}
    for c, cls in structs.items():
        assert got[(c, "size")] == ctypes.sizeof(cls), c
        for f, _ in cls._fields_:
            assert got[(c, f)] == getattr(cls, f).offset, (c, f)
    assert got[("group", "value")] == trit.KV4_GROUP and got[("most", "value")] == trit.MAX_TOP


def cache4(trit, **kw):  # noqa: F811
    a = dict(k=P, v=P, k_scale=P, v_scale=P, page_stride=5 * 64, head_stride=64, slot_stride=1, pages=10, heads=5,
             page_size=64, head_dim=128, reserved=0)
    a.update(kw)
    return trit.TritKv4Cache(**a)


BAD_CACHE = [(dict(k=NULL), ARG), (dict(v=NULL), ARG), (dict(k_scale=NULL), ARG), (dict(v_scale=NULL), ARG), (dict(k=ODD), ARG),
             (dict(v_scale=ODD), ARG), (dict(page_stride=-1), ARG), (dict(head_stride=-1), ARG), (dict(slot_stride=-1), ARG),
             (dict(reserved=1), ARG), (dict(head_dim=96), SHAPE), (dict(head_dim=32), SHAPE), (dict(pages=0), SHAPE),
             (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE), (dict(page_size=0), SHAPE)]


def refuses(fn, job, good, cases):
    """Each change of a sound job is refused with its status, and so are missing pointers."""
    for kw, code in cases:
        assert fn(ctypes.byref(job(**kw)), P, NULL) == code, kw
    assert fn(ctypes.byref(job()), NULL, NULL) == ARG
    assert fn(ctypes.byref(job()), BYTE, NULL) == ARG
    assert fn(None, P, NULL) == ARG


def test_append_refusals(trit):  # noqa: F811
    def job(**kw):
        a = dict(cache=cache4(trit), batch=batch(trit), q=P, k=P, v=P, q_out=P, starts=NULL, cos=P, sin=P, q_gain=NULL,
                 k_gain=NULL, q_stride=2560, k_stride=640, v_stride=640, rows=6, max_pos=1000, eps=1e-5, q_heads=20,
                 rot=128, src_dtype=0, dtype=1, flags=0)
        a.update(kw)
        return trit.TritKv4AppendJob(**a)
    cases = [(dict(cache=cache4(trit, **kw)), code) for kw, code in BAD_CACHE]
    cases += [(dict(batch=batch(trit, **kw)), code) for kw, code in BAD_BATCH]
    refuses(trit.lib().trit_kv4_append, job, None, cases + [
        (dict(k=NULL), ARG), (dict(v=NULL), ARG), (dict(q=NULL), ARG), (dict(q_out=NULL), ARG), (dict(cos=NULL), ARG),
        (dict(k=ODD), ARG), (dict(q_gain=ODD), ARG), (dict(sin=ODD), ARG), (dict(starts=BYTE, rows=5), ARG), (dict(flags=2), ARG),
        (dict(src_dtype=2), ARG), (dict(dtype=0), ARG), (dict(dtype=3), ARG), (dict(q_stride=2561), ARG),
        (dict(v_stride=-640), ARG), (dict(starts=P, batch=batch(trit, new_lens=P)), ARG), (dict(rot=136), SHAPE),
        (dict(rot=4), SHAPE), (dict(rot=-8), SHAPE), (dict(max_pos=-1), SHAPE), (dict(q_heads=21), SHAPE),
        (dict(q_heads=0), SHAPE), (dict(rows=5), SHAPE), (dict(rows=0, starts=P), SHAPE),
        (dict(rows=(1 << 24) + 1, starts=P), SHAPE), (dict(q_gain=P, eps=-1.0), SCALE), (dict(k_gain=P, eps=float("nan")), SCALE)])


def test_read_refusals(trit):  # noqa: F811
    def job(**kw):
        a = dict(cache=cache4(trit), batch=batch(trit), k=P, v=P, starts=P, rows=100, dtype=1, flags=0)
        a.update(kw)
        return trit.TritKv4ReadJob(**a)
    cases = [(dict(cache=cache4(trit, **kw)), code) for kw, code in BAD_CACHE]
    cases += [(dict(batch=batch(trit, **kw)), code) for kw, code in BAD_BATCH]
    refuses(trit.lib().trit_kv4_read, job, None, cases + [
        (dict(k=NULL), ARG), (dict(v=NULL), ARG), (dict(starts=NULL), ARG), (dict(k=ODD), ARG), (dict(starts=BYTE), ARG),
        (dict(dtype=0), ARG), (dict(flags=1), ARG), (dict(rows=0), SHAPE), (dict(rows=(1 << 27) + 1), SHAPE)])


def test_attn_refusals(trit):  # noqa: F811
    L = trit.lib()

    def job(**kw):
        a = dict(cache=cache4(trit), batch=batch(trit), q=P, out=P, lse=NULL, workspace=P, workspace_bytes=1 << 40,
                 q_stride=2560, scale=0.1, q_heads=20, dtype=1, out_dtype=0, flags=0, reserved=0)
        a.update(kw)
        return trit.TritAttn4Job(**a)
    need = L.trit_attn4_workspace_bytes(ctypes.byref(job()))
    assert need > 0 and L.trit_attn4_workspace_bytes(None) == -1
    sizes = [(dict(cache=cache4(trit, **kw)), code) for kw, code in BAD_CACHE]
    sizes += [(dict(batch=batch(trit, **kw)), code) for kw, code in BAD_BATCH]
    sizes += [(dict(dtype=0), ARG), (dict(out_dtype=2), ARG), (dict(flags=1), ARG), (dict(reserved=1), ARG),
              (dict(q_heads=21), SHAPE), (dict(q_heads=0), SHAPE), (dict(batch=batch(trit, B=4096, T=1 << 20)), SHAPE)]
    for kw, _ in sizes:
        assert L.trit_attn4_workspace_bytes(ctypes.byref(job(**kw))) == -1, kw
    refuses(L.trit_attn_paged4, job, None, sizes + [
        (dict(q=NULL), ARG), (dict(out=NULL), ARG), (dict(workspace=NULL), ARG), (dict(q=ODD), ARG), (dict(out=ODD), ARG),
        (dict(lse=ctypes.c_void_p(65538)), ARG), (dict(q_stride=2564), ARG), (dict(q_stride=-8), ARG),
        (dict(scale=float("inf")), SCALE), (dict(workspace_bytes=need - 1), 8)])


def test_prompt_refusals(trit):  # noqa: F811
    def job(**kw):
        a = dict(q=P, k=P, v=P, out=P, lse=NULL, q_starts=P, k_starts=NULL, q_stride=2560, k_stride=640, v_stride=640,
                 q_rows=100, k_rows=100, B=3, q_heads=20, heads=5, head_dim=128, dtype=1, out_dtype=1, scale=0.1, flags=0)
        a.update(kw)
        return trit.TritPromptJob(**a)
    refuses(trit.lib().trit_attn_prompt, job, None, [
        (dict(q=NULL), ARG), (dict(k=NULL), ARG), (dict(v=NULL), ARG), (dict(out=NULL), ARG), (dict(q_starts=NULL), ARG),
        (dict(q=ODD), ARG), (dict(v=ODD), ARG), (dict(out=ODD), ARG), (dict(lse=BYTE), ARG), (dict(q_starts=BYTE), ARG),
        (dict(k_starts=BYTE), ARG), (dict(dtype=0), ARG), (dict(dtype=3), ARG), (dict(out_dtype=2), ARG), (dict(flags=1), ARG),
        (dict(q_stride=2564), ARG), (dict(k_stride=632), ARG), (dict(v_stride=0), ARG), (dict(q_stride=1 << 38), ARG),
        (dict(head_dim=96), SHAPE), (dict(heads=0), SHAPE), (dict(q_heads=21), SHAPE), (dict(q_heads=0), SHAPE),
        (dict(B=0), SHAPE), (dict(B=4097), SHAPE), (dict(q_rows=0), SHAPE), (dict(k_rows=-1), SHAPE),
        (dict(k_rows=(1 << 27) + 1), SHAPE), (dict(q_rows=1 << 27), SHAPE), (dict(scale=0.0), SCALE), (dict(scale=-0.1), SCALE),
        (dict(scale=float("nan")), SCALE), (dict(scale=float("inf")), SCALE)])


def test_logprob_refusals(trit):  # noqa: F811
    def job(**kw):
        a = dict(logits=P, tokens=P, logprob=P, entropy=P, top_tokens=P, top_logprobs=P, stride=1000, rows=7, V=1000,
                 top_n=5, dtype=0, flags=0, reserved=0)
        a.update(kw)
        return trit.TritLogprobJob(**a)
    half = ctypes.c_void_p((1 << 16) + 2)
    refuses(trit.lib().trit_logprobs, job, None, [
        (dict(logits=NULL), ARG), (dict(tokens=NULL), ARG), (dict(logprob=NULL), ARG), (dict(top_tokens=NULL), ARG),
        (dict(top_logprobs=NULL), ARG), (dict(top_n=0), ARG), (dict(logits=half), ARG), (dict(entropy=half), ARG),
        (dict(logits=BYTE, dtype=1), ARG), (dict(dtype=3), ARG), (dict(flags=1), ARG), (dict(reserved=1), ARG),
        (dict(stride=-1), ARG), (dict(rows=0), SHAPE), (dict(rows=(1 << 24) + 1), SHAPE), (dict(V=0), SHAPE),
        (dict(V=1 << 31), SHAPE), (dict(top_n=65), SHAPE), (dict(top_n=-1, top_tokens=NULL, top_logprobs=NULL), SHAPE)])


def test_python_checks(trit):  # noqa: F811
    """CPU tensors, wrong types, shapes and layouts raise before anything is called."""
    torch = pytest.importorskip("torch")
    codes, pairs = torch.zeros(2, 5, 16, 64, dtype=torch.uint8), torch.zeros(2, 5, 16, 2, 2, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        trit.Kv4Cache(codes, codes, pairs, pairs)
    with pytest.raises(ValueError, match="pages"):
        trit.Kv4Cache(codes[0], codes, pairs, pairs)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rows, heads, D"):
        trit.PromptJob(x.flatten(1), x, x, x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        trit.PromptJob(x, x, x, x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="logits"):
        trit.LogprobJob(torch.zeros(4))
    with pytest.raises(ValueError, match="come together"):
        trit.LogprobJob(torch.zeros(4, 5), tokens=torch.zeros(4, dtype=torch.int32))


def test_a_stack_s_cache_has_4_or_16_bits():
    import bit_plane_select_gb300 as t
    from bit_plane_select_gb300.stack import ServedStack
    from test_served_stack_host import layer
    with pytest.raises(ValueError, match="cache_bits"):
        ServedStack([layer()], 64, t.Rope(), 4, 16, device="cpu", cache_bits=8)
    stack = ServedStack.__new__(ServedStack)
    stack.cache_bits = 16
    with pytest.raises(ValueError, match="4 bits"):
        stack.prompt_plan(None, 1, None, 1, None)
