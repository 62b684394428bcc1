"""The paged KV cache's refusals, without a device: the C entry points check
everything that does not lie in device memory before they touch one, and the
binding refuses tensors that the library would misread."""
import ctypes

import pytest
import torch

import block_discrete_diffusion_denoise_b200 as dg

A = 0x100000          # an aligned address, never dereferenced


@pytest.mark.parametrize("name", ["dg_paged_plan_args", "dg_paged_append_args", "dg_paged_attention_args"])
def test_argument_structs_match_the_header(name):
    import os
    import re
    src = open(os.path.join(os.path.dirname(__file__), "..", "include", "dg.h")).read()
    body = src[src.index("typedef struct %s {" % name):src.index("} %s;" % name)]
    fields = re.findall(r"(const void\*|const int32_t\*|const float\*|int32_t\*|void\*|float\*|int64_t|int32_t|float)"
                        r"\s+([a-z_]+);", body)
    want = [(n, {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float}.get(t, ctypes.c_void_p))
            for t, n in fields]
    assert want == list(getattr(dg, name)._fields_)


@pytest.mark.parametrize("packer,name", [(dg._PAGED_PLAN_ARGS, "dg_paged_plan_args"),
                                         (dg._PAGED_APPEND_ARGS, "dg_paged_append_args"),
                                         (dg._PAGED_ATTENTION_ARGS, "dg_paged_attention_args")])
def test_packed_arguments_match_the_structs(packer, name):
    """the binding packs the argument structs without building the ctypes objects"""
    cls = getattr(dg, name)
    values = [0.5 if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
    packed = packer.pack(*values)
    assert len(packed) == ctypes.sizeof(cls)
    s = cls.from_buffer_copy(packed)
    assert [getattr(s, n) for n, _ in cls._fields_] == values


def plan(**kw):
    a = dict(cached=A, new=A + 0x1000, batch=3, table=A + 0x2000, width=8, stride=8, ring=A + 0x3000, n_pages=100,
             state=A + 0x4000, page=64, cu=A + 0x5000, kv=A + 0x6000, pos=A + 0x7000, slots=A + 0x8000, cap=10,
             out=A + 0x9000)
    a.update(kw)
    args = dg.dg_paged_plan_args(a["cached"], a["new"], a["table"], a["ring"], a["state"], a["cu"], a["kv"], a["pos"],
                                 a["slots"], a["out"], a["stride"], a["batch"], a["width"], a["n_pages"], a["page"],
                                 a["cap"])
    return dg.load_library().dg_paged_plan(ctypes.byref(args), None)


@pytest.mark.parametrize("kw,status", [
    (dict(cached=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(ring=None), 1), (dict(state=None), 1),
    (dict(cu=None), 1), (dict(kv=None), 1), (dict(out=None), 1), (dict(pos=None), 1), (dict(slots=None), 1),
    (dict(batch=0), 1), (dict(batch=-1), 1), (dict(width=0), 1), (dict(stride=7), 1), (dict(n_pages=0), 1),
    (dict(cap=-1), 1), (dict(out=A + 0x4000), 1), (dict(kv=A), 1), (dict(kv=A + 0x1000), 1),
    (dict(out=A + 0x4000 - 8), 1), (dict(slots=A + 0x7000), 1), (dict(slots=A + 0x7000 + 36), 1), (dict(cu=A + 8), 1),
    (dict(ring=A + 0x2000 + 4 * 23), 1), (dict(pos=A + 0x3000 + 4 * 99), 1),
    (dict(page=0), 7), (dict(page=48), 7), (dict(page=256), 7), (dict(n_pages=2 ** 31 // 64), 3),
])
def test_plan_refuses(kw, status):
    assert plan(**kw) == status


def append(**kw):
    a = dict(qkv=A, stride=5632, rows=4, hq=16, hkv=8, d=176, pos=A + 0x20000, slots=A + 0x21000, rope=A + 0x22000,
             n_pos=100, k=A + 0x1000000, v=A + 0x2000000, n_pages=10, page=64, q=A + 0x40000)
    a.update(kw)
    args = dg.dg_paged_append_args(a["qkv"], a["pos"], a["slots"], a["rope"], a["k"], a["v"], a["q"], a["stride"],
                                   a["rows"], a["hq"], a["hkv"], a["d"], a["n_pos"], a["n_pages"], a["page"])
    return dg.load_library().dg_paged_append(ctypes.byref(args), None)


@pytest.mark.parametrize("kw,status", [
    (dict(qkv=None), 1), (dict(pos=None), 1), (dict(slots=None), 1), (dict(rope=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(q=None), 1), (dict(rows=-1), 1), (dict(n_pos=0), 1), (dict(n_pages=0), 1),
    (dict(qkv=A + 8), 1), (dict(rope=A + 4), 1), (dict(k=A + 2), 1), (dict(v=A + 8), 1), (dict(q=A + 8), 1),
    (dict(stride=5631), 1), (dict(stride=5636), 1), (dict(hq=0), 1), (dict(d=96, stride=5632), 7), (dict(hkv=3), 7),
    (dict(hq=24, stride=8000), 7), (dict(page=17), 7), (dict(n_pages=2 ** 25), 3), (dict(rows=0), 0),
    (dict(q=A), 1), (dict(q=A + 4 * 5632 * 2 - 16), 1), (dict(v=A + 0x1000000), 1), (dict(k=A + 0x20000), 1),
    (dict(v=A + 0x1000000 + 10 * 64 * 8 * 176 * 2 - 16), 1),
])
def test_append_refuses(kw, status):
    assert append(**kw) == status


def attention(**kw):
    a = dict(q=A, k_pages=A, v_pages=A, block_table=A, kv_lens=A, cu_rows=A, out=A, lse=None, workspace=None,
             workspace_bytes=0, q_stride=2816,
             table_stride=8, n_rows=4, batch=2, n_q_heads=16, n_kv_heads=8, head_dim=176, n_pages=10, page_size=64,
             table_width=8, causal=0, max_rows=0, scale=0.1)
    a.update(kw)
    return dg.load_library().dg_paged_attention(ctypes.byref(dg.dg_paged_attention_args(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(block_table=None), 1),
    (dict(kv_lens=None), 1), (dict(cu_rows=None), 1), (dict(out=None), 1), (dict(n_rows=-1), 1), (dict(batch=0), 1),
    (dict(n_pages=0), 1), (dict(table_width=0), 1), (dict(table_stride=7), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=A + 8), 1),
    (dict(k_pages=A + 8), 1), (dict(v_pages=A + 8), 1), (dict(out=A + 8), 1), (dict(q_stride=2815), 1),
    (dict(q_stride=2820), 1), (dict(n_q_heads=0), 1), (dict(head_dim=80), 7), (dict(n_q_heads=17), 7),
    (dict(n_q_heads=24, q_stride=8000), 7), (dict(page_size=8), 7), (dict(n_pages=2 ** 25), 3),
    (dict(n_pages=2 ** 23), 3), (dict(table_width=2 ** 25, table_stride=2 ** 25), 3), (dict(n_rows=0), 0),
    (dict(), 1), (dict(workspace=A + 8, workspace_bytes=2 ** 40), 1),
])
def test_attention_refuses(kw, status):
    assert attention(**kw) == status


@pytest.mark.parametrize("name", ["dg_paged_plan", "dg_paged_append", "dg_paged_attention"])
def test_no_arguments_are_refused(name):
    assert getattr(dg.load_library(), name)(None, None) == dg.DG_ERR_INVALID_ARG


def refused(fn, *a, **kw):
    with pytest.raises(dg.DGError) as e:
        fn(*a, **kw)
    assert e.value.status == dg.DG_ERR_INVALID_ARG


def test_the_binding_refuses_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    b = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    refused(dg.paged_plan, i, i, i.view(2, 2), i, i, 16, i, i, i, i, i)
    refused(dg.paged_append, b.view(4, -1), i, i, torch.zeros(4, 32, 2), pool, pool, b)
    refused(dg.paged_attention, b, pool, pool, i.view(2, 2), i, i, b)
    refused(dg.paged_attention, None, pool, pool, i.view(2, 2), i, i, b)
    refused(dg.paged_plan, None, i, None, i, i, 16, i, i, i, i, i)
