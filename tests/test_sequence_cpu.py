"""The sequence operators' C ABI without a GPU: layouts, workspace sizes, and
argument errors, which come back before any device work."""
import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20   # stands for a device pointer, 256-byte aligned: nothing below reads it


@pytest.fixture(scope="module")
def lib():
    from dynamic_embedding_tables_amd import recis
    recis.load_library()
    return recis


def test_attn_desc_layout(lib, tmp_path):
    cls = lib.recis_attn_desc
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "recis.h"', "int main(void){",
             'printf("size %zu\\n", sizeof(recis_attn_desc));']
    lines += [f'printf("{f[0]} %zu\\n", offsetof(recis_attn_desc, {f[0]}));' for f in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.check_call(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                           "/opt/rocm/include", str(src), "-o", str(exe)])
    got = dict(line.split() for line in subprocess.check_output([str(exe)], text=True).splitlines())
    assert int(got.pop("size")) == C.sizeof(cls)
    for name, at in got.items():
        assert getattr(cls, name).offset == int(at), name


def test_workspace_sizes(lib):
    L = lib.load_library()
    assert L.recis_embed_bwd_workspace_bytes(0, 1, 1) > 0
    assert L.recis_embed_bwd_workspace_bytes(1000, 100, 64) < L.recis_embed_bwd_workspace_bytes(100000, 100, 64)
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 31, 1, 1), (1, (1 << 30) + 1, 1), (1, 1, (1 << 16) + 1)):
        assert L.recis_embed_bwd_workspace_bytes(*bad) == -1, bad
    assert L.recis_layernorm_bwd_workspace_bytes(10, 64) > 0
    for bad in ((-1, 1), (1, 0), (1, 16385)):
        assert L.recis_layernorm_bwd_workspace_bytes(*bad) == -1, bad


EMBED_FWD = dict(tokens=P, n=4, weight=P, dtype=0, rows=10, dim=8, weight_stride=8, scale=1.0, out=P, out_stride=8,
                 error=None, stream=None)
EMBED_BWD = dict(tokens=P, n=4, grad_out=P, grad_dtype=0, grad_stride=8, rows=10, dim=8, scale=1.0, grad_weight=P,
                 weight_dtype=0, weight_stride=8, workspace=P, workspace_bytes=1 << 40, error=None, stream=None)
NORM_FWD = dict(x=P, dtype=0, x_stride=8, m=4, dim=8, weight=None, bias=None, weight_dtype=0, eps=1e-5, y=P, y_stride=8,
                mean=P, rstd=P, stream=None)
NORM_BWD = dict(grad_y=P, grad_stride=8, x=P, x_stride=8, dtype=0, m=4, dim=8, mean=P, rstd=P, weight=None,
                weight_dtype=0, grad_x=P, grad_x_stride=8, grad_weight=P, grad_bias=P, workspace=P,
                workspace_bytes=1 << 40, stream=None)
INVALID, UNSUPPORTED = 1, 6


@pytest.mark.parametrize("name,args,change,status", [
    ("recis_embed_fwd", EMBED_FWD, c, s) for c, s in (
        (dict(dtype=2), INVALID), (dict(n=-1), INVALID), (dict(rows=0), INVALID), (dict(dim=0), INVALID),
        (dict(weight_stride=7), INVALID), (dict(out_stride=7), INVALID), (dict(tokens=None), INVALID),
        (dict(weight=None), INVALID), (dict(out=None), INVALID), (dict(tokens=P + 4), INVALID),
        (dict(weight=P + 2), INVALID), (dict(error=P + 1), INVALID), (dict(n=1 << 31), UNSUPPORTED),
        (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(dim=1 << 17, weight_stride=1 << 17, out_stride=1 << 17), UNSUPPORTED))
] + [
    ("recis_embed_bwd", EMBED_BWD, c, s) for c, s in (
        (dict(grad_dtype=-1), INVALID), (dict(weight_dtype=2), INVALID), (dict(n=-1), INVALID), (dict(rows=0), INVALID),
        (dict(dim=0), INVALID), (dict(grad_stride=7), INVALID), (dict(weight_stride=7), INVALID),
        (dict(tokens=None), INVALID), (dict(grad_out=None), INVALID), (dict(grad_weight=None), INVALID),
        (dict(workspace=None), INVALID), (dict(workspace=P + 16), INVALID), (dict(workspace_bytes=64), INVALID),
        (dict(grad_out=P + 1), INVALID), (dict(n=1 << 31), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED))
] + [
    ("recis_layernorm_fwd", NORM_FWD, c, s) for c, s in (
        (dict(dtype=3), INVALID), (dict(weight_dtype=9), INVALID), (dict(m=-1), INVALID), (dict(dim=0), INVALID),
        (dict(x_stride=7), INVALID), (dict(y_stride=7), INVALID), (dict(eps=-1.0), INVALID),
        (dict(eps=float("nan")), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(x=None), INVALID),
        (dict(y=None), INVALID), (dict(x=P + 2), INVALID), (dict(weight=P + 2), INVALID),
        (dict(dim=16385, x_stride=16385, y_stride=16385), UNSUPPORTED))
] + [
    ("recis_layernorm_bwd", NORM_BWD, c, s) for c, s in (
        (dict(dtype=3), INVALID), (dict(weight_dtype=9), INVALID), (dict(m=-1), INVALID), (dict(dim=0), INVALID),
        (dict(x_stride=7), INVALID), (dict(grad_stride=7), INVALID), (dict(grad_x_stride=7), INVALID),
        (dict(grad_y=None), INVALID), (dict(x=None), INVALID), (dict(grad_x=None), INVALID), (dict(mean=None), INVALID),
        (dict(rstd=None), INVALID), (dict(workspace=None), INVALID), (dict(workspace=P + 4), INVALID),
        (dict(workspace_bytes=63), INVALID), (dict(grad_x=P + 1), INVALID),
        (dict(dim=16385, x_stride=16385, grad_stride=16385, grad_x_stride=16385), UNSUPPORTED))
])
def test_rows_are_refused(lib, name, args, change, status):
    assert getattr(lib.load_library(), name)(*{**args, **change}.values()) == status


def desc(lib, **change):
    d = lib.recis_attn_desc()
    d.dtype, d.batch, d.q_len, d.kv_len, d.q_heads, d.kv_heads, d.head_dim, d.scale = 0, 2, 3, 5, 4, 2, 8, 0.5
    for name in ("q_strides", "k_strides", "v_strides", "o_strides", "do_strides", "dq_strides", "dk_strides", "dv_strides"):
        getattr(d, name)[:] = (160, 32, 8)
    for name, value in change.items():
        setattr(d, name, value)
    return d


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), INVALID), (dict(batch=-1), INVALID), (dict(q_len=-1), INVALID), (dict(kv_len=-1), INVALID),
    (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(head_dim=0), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(kv_offsets=P, kv_lens=P), INVALID), (dict(kv_offsets=P, kv_rows=-1), INVALID),
    (dict(kv_lens=P + 2), INVALID), (dict(kv_offsets=P + 1), INVALID), (dict(error=P + 3), INVALID),
    (dict(head_dim=129), UNSUPPORTED), (dict(kv_len=(1 << 30) + 1), UNSUPPORTED), (dict(batch=1 << 24), UNSUPPORTED),
])
def test_attention_descriptions_are_refused(lib, change, status):
    L, d = lib.load_library(), desc(lib, **change)
    assert L.recis_cross_attn_fwd(C.byref(d), P, P, P, P, P, P, 1 << 40, None) == status
    assert L.recis_cross_attn_bwd(C.byref(d), P, P, P, P, P, P, P, P, P, P, 1 << 40, None) == status
    for backward in (0, 1):
        assert L.recis_cross_attn_workspace_bytes(C.byref(d), backward) == -1


def test_attention_pointers_are_refused(lib):
    L, d = lib.load_library(), desc(lib, kv_len=100000, q_len=1)
    need = [L.recis_cross_attn_workspace_bytes(C.byref(d), b) for b in (0, 1)]
    assert need[0] > 0 and need[1] > 0   # one query over many keys: the keys are split
    assert L.recis_cross_attn_workspace_bytes(None, 0) == -1
    assert L.recis_cross_attn_fwd(None, P, P, P, P, P, P, 1 << 40, None) == INVALID
    fwd, bwd = [P] * 6, [P] * 10
    for i, bad in [(i, None) for i in range(4)] + [(0, P + 2), (3, P + 1), (4, P + 2), (5, None), (5, P + 128)]:
        args = fwd[:i] + [bad] + fwd[i + 1:]
        assert L.recis_cross_attn_fwd(C.byref(d), *args, need[0], None) == INVALID, (i, bad)
    assert L.recis_cross_attn_fwd(C.byref(d), *fwd, need[0] - 1, None) == INVALID
    for i, bad in [(i, None) for i in range(10)] + [(0, P + 2), (8, P + 1), (5, P + 2), (9, P + 128)]:
        args = bwd[:i] + [bad] + bwd[i + 1:]
        assert L.recis_cross_attn_bwd(C.byref(d), *args, need[1], None) == INVALID, (i, bad)
    assert L.recis_cross_attn_bwd(C.byref(d), *bwd, need[1] - 1, None) == INVALID


def test_nothing_to_do_is_no_error(lib):
    L = lib.load_library()
    assert L.recis_embed_fwd(*{**EMBED_FWD, **dict(n=0, tokens=None, out=None)}.values()) == 0
    assert L.recis_layernorm_fwd(*{**NORM_FWD, **dict(m=0, x=None, y=None)}.values()) == 0
    d = desc(lib, batch=0)
    assert L.recis_cross_attn_fwd(C.byref(d), None, None, None, None, None, None, 0, None) == 0
    assert L.recis_cross_attn_bwd(C.byref(d), *[None] * 10, 0, None) == 0


# Sizes past the C ABI's 32-bit integers are refused as the ABI refuses large ones, not taken by their low 32 bits.
WIDE = [(1 << 31) + 64, (1 << 32) + 64, 1 << 40]


@pytest.mark.parametrize("size", WIDE)
def test_sizes_past_32_bits_have_no_workspace(lib, size):
    assert lib.recis_layernorm_bwd_workspace_bytes(4, size) == -1
    assert lib.recis_embed_bwd_workspace_bytes(4, 10, size) == -1
    d = desc(lib)
    d.kv_len = lib.int32(size)
    assert lib.recis_cross_attn_workspace_bytes(d, True) == -1


@pytest.mark.parametrize("size", WIDE)
def test_rows_past_32_bits_are_refused(lib, size):
    import torch
    t, stream = torch.zeros(64), type("Stream", (), {"cuda_stream": None})
    for call in (lambda: lib.recis_embed_fwd(t, 4, t, 0, 10, size, size, 1.0, t, size, stream=stream),
                 lambda: lib.recis_embed_bwd(t, 4, t, 0, size, 10, size, 1.0, t, 0, size, t, 1 << 40, stream=stream),
                 lambda: lib.recis_layernorm_fwd(t, 0, size, 4, size, None, None, 0, 1e-5, t, size, stream=stream),
                 lambda: lib.recis_layernorm_bwd(t, size, t, size, 0, 4, size, t, t, None, 0, t, size, t, t, t, 1 << 40,
                                                 stream=stream)):
        with pytest.raises(lib.RecisError) as e:
            call()
        assert e.value.status == UNSUPPORTED


@pytest.mark.parametrize("most,status", [(size, UNSUPPORTED) for size in WIDE] + [(-(1 << 32) + 5, INVALID)])
def test_key_counts_past_32_bits_are_refused(lib, most, status):
    import torch

    from dynamic_embedding_tables_amd import sequence
    q, k, offsets = torch.zeros(2, 3, 2, 8), torch.zeros(9, 2, 8), torch.tensor([0, 4, 9], dtype=torch.int32)
    d, _ = sequence._attn_desc(q, k, k, None, offsets, None, most, None, None)
    L = lib.load_library()
    assert L.recis_cross_attn_fwd(C.byref(d), P, P, P, P, P, P, 1 << 40, None) == status
    assert L.recis_cross_attn_bwd(C.byref(d), P, P, P, P, P, P, P, P, P, P, 1 << 40, None) == status


def test_sizes_past_a_launch_are_refused(lib):
    """2^23 pairs of (entry, key head): 255 tiles of 64 keys can be launched for their gradients, 256 cannot."""
    L = lib.load_library()
    d = desc(lib, batch=1 << 20, q_heads=8, kv_heads=8, q_len=1, kv_len=255 * 64)
    assert L.recis_cross_attn_workspace_bytes(C.byref(d), 0) == 0
    assert L.recis_cross_attn_workspace_bytes(C.byref(d), 1) > 0
    d.kv_len += 1
    assert L.recis_cross_attn_workspace_bytes(C.byref(d), 0) == 0
    assert L.recis_cross_attn_workspace_bytes(C.byref(d), 1) == -1
    assert L.recis_cross_attn_bwd(C.byref(d), *[P] * 10, 1 << 60, None) == UNSUPPORTED
    d.q_len, d.kv_len = 255 * 64 + 1, 5
    for backward in (0, 1):
        assert L.recis_cross_attn_workspace_bytes(C.byref(d), backward) == -1
    assert L.recis_cross_attn_fwd(C.byref(d), *[P] * 6, 1 << 60, None) == UNSUPPORTED
    assert L.recis_cross_attn_bwd(C.byref(d), *[P] * 10, 1 << 60, None) == UNSUPPORTED
    many = dict(n=1 << 25, dim=(1 << 15) + 1, weight_stride=1 << 16, out_stride=1 << 16)
    assert L.recis_embed_fwd(*{**EMBED_FWD, **many}.values()) == UNSUPPORTED


def test_empty_head_vectors_are_refused(lib):
    import torch

    from dynamic_embedding_tables_amd import sequence
    q, k = torch.zeros(2, 3, 2, 0), torch.zeros(2, 5, 2, 0)
    d, _ = sequence._attn_desc(q, k, k, None, None, None, None, None, None)
    assert lib.load_library().recis_cross_attn_fwd(C.byref(d), P, P, P, P, P, P, 1 << 40, None) == INVALID
