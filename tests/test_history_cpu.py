"""The C ABI of the operators of a growing history without a GPU: layouts, workspace sizes, frequencies, and argument
errors, which come back before any device work."""
import ctypes as C
import math
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20   # stands for a device pointer, 256-byte aligned: nothing below reads it
INVALID, UNSUPPORTED = 1, 6


@pytest.fixture(scope="module")
def lib():
    from dynamic_embedding_tables_amd import recis
    recis.load_library()
    return recis


@pytest.mark.parametrize("name", ["recis_rotary_desc", "recis_append_desc", "recis_paged_attn_desc",
                                  "recis_self_attn_desc"])
def test_desc_layouts(lib, tmp_path, name):
    cls = getattr(lib, name)
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "recis.h"', "int main(void){",
             f'printf("size %zu\\n", sizeof({name}));']
    lines += [f'printf("{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.check_call(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                           "/opt/rocm/include", str(src), "-o", str(exe)])
    got = dict(line.split() for line in subprocess.check_output([str(exe)], text=True).splitlines())
    assert int(got.pop("size")) == C.sizeof(cls)
    for field, at in got.items():
        assert getattr(cls, field).offset == int(at), field


@pytest.mark.parametrize("name", ["rotary", "append", "paged_attn", "self_attn"])
def test_packed_descriptions_are_the_structures(lib, name):
    cls = getattr(lib, f"recis_{name}_desc")
    d, values = cls(), []
    for i, (field, kind) in enumerate(cls._fields_):
        if hasattr(kind, "_length_"):
            value = [1000 * i + j for j in range(kind._length_)]
            getattr(d, field)[:] = value
            values += value
        else:
            setattr(d, field, i + 1)
            values.append(i + 1)
    assert getattr(lib, f"pack_{name}_desc")(*values) == bytes(d)


def described(cls, values, **change):
    d = cls()
    for name, value in {**values, **change}.items():
        if isinstance(value, tuple):
            getattr(d, name)[:] = value
        else:
            setattr(d, name, value)
    return d


S3 = (160, 32, 8)
ROTARY = dict(dtype=0, heads=2, head_dim=8, rot_dim=8, interleaved=0, amplitude=1.0, batch=2, seq=3, freqs=P,
              positions=None, pos_strides=(0, 1), x_strides=S3, out_strides=S3)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), INVALID), (dict(heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(rot_dim=3), INVALID),
    (dict(rot_dim=10), INVALID), (dict(rot_dim=-2), INVALID), (dict(amplitude=math.inf), INVALID),
    (dict(amplitude=math.nan), INVALID), (dict(batch=-1), INVALID), (dict(seq=-1), INVALID), (dict(freqs=None), INVALID),
    (dict(freqs=P + 4), INVALID), (dict(positions=P + 4), INVALID), (dict(head_dim=1025), UNSUPPORTED),
    (dict(heads=1 << 16), UNSUPPORTED), (dict(batch=1 << 41), UNSUPPORTED), (dict(batch=1 << 30, seq=1 << 30), UNSUPPORTED),
    (dict(batch=1 << 40, seq=1, heads=1000), UNSUPPORTED),
])
def test_rotary_descriptions_are_refused(lib, change, status):
    L = lib.load_library()
    d = described(lib.recis_rotary_desc, ROTARY, **change)
    for backward in (0, 1):
        assert L.recis_rotary(C.byref(d), backward, P, P, None) == status


def test_rotary_pointers_are_refused(lib):
    L, d = lib.load_library(), described(lib.recis_rotary_desc, ROTARY)
    assert L.recis_rotary(None, 0, P, P, None) == INVALID
    for x, out in ((None, P), (P, None), (P + 2, P), (P, P + 2)):
        assert L.recis_rotary(C.byref(d), 0, x, out, None) == INVALID
    for none in (dict(batch=0), dict(seq=0)):
        assert L.recis_rotary(C.byref(described(lib.recis_rotary_desc, ROTARY, **none)), 0, None, None, None) == 0
    still = described(lib.recis_rotary_desc, ROTARY, rot_dim=0, freqs=None)
    assert L.recis_rotary(C.byref(still), 0, P, P, None) == 0   # in place with nothing that turns: no work


APPEND = dict(dtype=0, batch=2, new_len=3, q_heads=2, kv_heads=2, head_dim=8, rot_dim=8, interleaved=0, amplitude=1.0,
              page_size=4, table_width=5, pages=9, table_stride=5, rows=0, q_strides=S3, q_out_strides=S3, k_strides=S3,
              v_strides=S3, k_cache_strides=S3, v_cache_strides=S3, freqs=P, q_offsets=None, kv_lens=P, page_table=P,
              error=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=-1), INVALID), (dict(batch=-1), INVALID), (dict(new_len=-1), INVALID), (dict(q_heads=-1), INVALID),
    (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(rot_dim=9), INVALID), (dict(amplitude=math.nan), INVALID),
    (dict(page_size=0), INVALID), (dict(pages=-1), INVALID), (dict(table_width=-1), INVALID), (dict(table_stride=4), INVALID),
    (dict(freqs=None), INVALID), (dict(kv_lens=None), INVALID), (dict(kv_lens=P + 2), INVALID), (dict(q_offsets=P + 1), INVALID),
    (dict(q_offsets=P, rows=-1), INVALID), (dict(page_table=P + 2), INVALID), (dict(page_table=None), INVALID),
    (dict(error=P + 1), INVALID), (dict(head_dim=1025), UNSUPPORTED), (dict(q_heads=1 << 15), UNSUPPORTED),
    (dict(page_size=1 << 28, table_stride=1 << 20), UNSUPPORTED), (dict(pages=(1 << 31) + 1), UNSUPPORTED),
    (dict(q_offsets=P, rows=(1 << 31) + 1), UNSUPPORTED),
])
def test_append_descriptions_are_refused(lib, change, status):
    d = described(lib.recis_append_desc, APPEND, **change)
    assert lib.load_library().recis_cache_append(C.byref(d), P, P, P, P, P, P, None) == status


def test_append_pointers_are_refused(lib):
    L, d = lib.load_library(), described(lib.recis_append_desc, APPEND)
    assert L.recis_cache_append(None, P, P, P, P, P, P, None) == INVALID
    for i in range(6):
        for bad in (None, P + 2):
            args = [P] * 6
            args[i] = bad
            assert L.recis_cache_append(C.byref(d), *args, None) == INVALID, (i, bad)
    for none in (dict(batch=0), dict(new_len=0), dict(q_offsets=P, rows=0)):
        assert L.recis_cache_append(C.byref(described(lib.recis_append_desc, APPEND, **none)), *[None] * 6, None) == 0


PAGED = dict(dtype=0, batch=2, q_len=3, q_heads=4, kv_heads=2, head_dim=8, causal=1, window=0, sinks=0, page_size=4,
             table_width=5, scale=0.5, pages=9, table_stride=5, q_rows=0, q_strides=S3, o_strides=S3, k_strides=S3,
             v_strides=S3, q_offsets=None, kv_lens=P, page_table=P, error=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), INVALID), (dict(batch=-1), INVALID), (dict(q_len=-1), INVALID), (dict(q_heads=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(head_dim=0), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(causal=0, window=3), INVALID), (dict(page_size=0), INVALID), (dict(pages=-1), INVALID), (dict(table_width=-1), INVALID),
    (dict(table_stride=4), INVALID), (dict(q_offsets=P, q_rows=-1), INVALID), (dict(q_offsets=P + 2), INVALID),
    (dict(kv_lens=P + 1), INVALID), (dict(page_table=P + 3), INVALID), (dict(error=P + 2), INVALID),
    (dict(head_dim=129), UNSUPPORTED), (dict(page_size=1 << 28), UNSUPPORTED), (dict(pages=(1 << 31) + 1), UNSUPPORTED),
    (dict(q_len=(1 << 29) + 1), UNSUPPORTED), (dict(batch=1 << 24), UNSUPPORTED),
    (dict(batch=1 << 23, q_len=1 << 20, kv_heads=2), UNSUPPORTED),
])
def test_paged_descriptions_are_refused(lib, change, status):
    L, d = lib.load_library(), described(lib.recis_paged_attn_desc, PAGED, **change)
    assert L.recis_paged_attn_fwd(C.byref(d), P, P, P, P, P, P, 1 << 60, None) == status
    assert L.recis_paged_attn_workspace_bytes(C.byref(d)) == -1


def test_paged_pointers_are_refused(lib):
    L, d = lib.load_library(), described(lib.recis_paged_attn_desc, PAGED, q_len=1, table_width=5000, table_stride=5000)
    need = L.recis_paged_attn_workspace_bytes(C.byref(d))
    assert need > 0   # few rows over many keys: the keys are split
    assert L.recis_paged_attn_fwd(None, P, P, P, P, P, P, need, None) == INVALID
    for i, bad in [(i, None) for i in (0, 1, 2, 3, 5)] + [(0, P + 2), (1, P + 1), (2, P + 2), (3, P + 2), (4, P + 2), (5, P + 16)]:
        args = [P] * 6
        args[i] = bad
        assert L.recis_paged_attn_fwd(C.byref(d), *args, need, None) == INVALID, (i, bad)
    assert L.recis_paged_attn_fwd(C.byref(d), *[P] * 6, need - 1, None) == INVALID
    for change in (dict(kv_lens=None), dict(page_table=None)):
        assert L.recis_paged_attn_fwd(C.byref(described(lib.recis_paged_attn_desc, PAGED, **change)), *[P] * 6, 1 << 60,
                                      None) == INVALID
    for none in (dict(batch=0), dict(q_len=0), dict(q_offsets=P, q_rows=0)):
        e = described(lib.recis_paged_attn_desc, PAGED, **none)
        assert L.recis_paged_attn_fwd(C.byref(e), *[None] * 6, 0, None) == 0


SELF = dict(dtype=0, batch=2, len=5, q_heads=4, kv_heads=2, head_dim=8, window=0, sinks=0, scale=0.5, rows=0, q_strides=S3,
            k_strides=S3, v_strides=S3, o_strides=S3, do_strides=S3, dq_strides=S3, dk_strides=S3, dv_strides=S3, lens=None,
            offsets=None, kv_mask=None, mask_stride=0, error=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), INVALID), (dict(batch=-1), INVALID), (dict(len=-1), INVALID), (dict(q_heads=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(head_dim=0), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(offsets=P, lens=P), INVALID), (dict(offsets=P, rows=-1), INVALID), (dict(lens=P + 2), INVALID),
    (dict(offsets=P + 2), INVALID), (dict(error=P + 1), INVALID), (dict(head_dim=129), UNSUPPORTED),
    (dict(len=(1 << 29) + 1), UNSUPPORTED), (dict(batch=1 << 24), UNSUPPORTED), (dict(batch=1 << 23, len=1 << 20), UNSUPPORTED),
])
def test_self_descriptions_are_refused(lib, change, status):
    L, d = lib.load_library(), described(lib.recis_self_attn_desc, SELF, **change)
    assert L.recis_self_attn_fwd(C.byref(d), P, P, P, P, P, P, 1 << 60, None) == status
    assert L.recis_self_attn_bwd(C.byref(d), *[P] * 10, 1 << 60, None) == status
    for backward in (0, 1):
        assert L.recis_self_attn_workspace_bytes(C.byref(d), backward) == -1


def test_self_pointers_are_refused(lib):
    L, d = lib.load_library(), described(lib.recis_self_attn_desc, SELF, batch=1, len=4000, window=300, sinks=4)
    need = [L.recis_self_attn_workspace_bytes(C.byref(d), b) for b in (0, 1)]
    assert need[0] > 0 and need[1] > 0   # few histories: the keys are split
    assert L.recis_self_attn_fwd(None, *[P] * 6, need[0], None) == INVALID
    assert L.recis_self_attn_bwd(None, *[P] * 10, need[1], None) == INVALID
    for i, bad in [(i, None) for i in (0, 1, 2, 3, 5)] + [(0, P + 2), (3, P + 1), (4, P + 2), (5, P + 128)]:
        args = [P] * 6
        args[i] = bad
        assert L.recis_self_attn_fwd(C.byref(d), *args, need[0], None) == INVALID, (i, bad)
    for i, bad in [(i, None) for i in range(10)] + [(0, P + 2), (5, P + 1), (8, P + 1), (9, P + 128)]:
        args = [P] * 10
        args[i] = bad
        assert L.recis_self_attn_bwd(C.byref(d), *args, need[1], None) == INVALID, (i, bad)
    assert L.recis_self_attn_fwd(C.byref(d), *[P] * 6, need[0] - 1, None) == INVALID
    assert L.recis_self_attn_bwd(C.byref(d), *[P] * 10, need[1] - 1, None) == INVALID
    for none in (dict(batch=0), dict(len=0)):
        e = described(lib.recis_self_attn_desc, SELF, **none)
        assert L.recis_self_attn_fwd(C.byref(e), *[None] * 6, 0, None) == 0
        assert L.recis_self_attn_bwd(C.byref(e), *[None] * 10, 0, None) == 0


def test_frequencies():
    from dynamic_embedding_tables_amd.sequence import rotary_frequencies

    def f(*args, **kw):
        return rotary_frequencies(*args, device="cpu", **kw)

    assert f(0).numel() == 0
    assert torch.equal(f(8), torch.tensor([10000.0 ** (-i / 4) for i in range(4)], dtype=torch.float64))
    assert torch.equal(f(8, scaling="linear", factor=4.0), f(8) / 4)
    scaled = f(8, scaling="base", factor=4.0)
    assert scaled[0] == 1 and abs(float(scaled[-1] / f(8)[-1]) - 0.25) < 1e-12
    base = f(64)
    turns = 1000 * base / (2 * math.pi)
    parts = f(64, scaling="parts", factor=8.0, original_len=1000)
    assert torch.equal(parts[turns >= 4], base[turns >= 4])
    assert torch.allclose(parts[turns <= 1], base[turns <= 1] / 8, rtol=1e-15, atol=0)
    middle = (turns > 1) & (turns < 4)
    w = (turns[middle] - 1) / 3
    assert bool(middle.any()) and torch.allclose(parts[middle], w * base[middle] + (1 - w) * base[middle] / 8, rtol=1e-14, atol=0)
    for bad in (dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=8, scaling="other"), dict(rot_dim=8, factor=0.0),
                dict(rot_dim=2, scaling="base", factor=2.0), dict(rot_dim=8, scaling="parts"),
                dict(rot_dim=8, scaling="parts", original_len=100, slow=4.0, fast=4.0), dict(rot_dim=8, base=-1.0)):
        with pytest.raises(ValueError):
            f(**bad)


# Sizes past the C ABI's 32-bit integers are refused as the ABI refuses large ones, not taken by their low 32 bits.
@pytest.mark.parametrize("size", [(1 << 31) + 64, (1 << 32) + 64, 1 << 40])
def test_sizes_past_32_bits_are_refused(lib, size):
    from dynamic_embedding_tables_amd import sequence
    q, off = torch.zeros(10, 2, 8), torch.tensor([0, 4, 10], dtype=torch.int32)
    head, tail, *_ = sequence._self_desc(q, q, q, None, off, None, size, None, 0, None, None)
    d = lib.pack_self_attn_desc(*head, *[0] * 15, *tail)
    assert lib.recis_self_attn_workspace_bytes(d, True) == -1
    assert lib.load_library().recis_self_attn_fwd(d, *[P] * 6, 1 << 60, None) == UNSUPPORTED
    window, sinks = sequence._band(size, size)
    assert window == (1 << 31) - 1 and sinks == (1 << 31) - 1   # more than any length


def test_shifts_that_find_a_page(lib):
    """The division of a position by the page size, as the kernels do it, for positions at the ends of pages."""
    for page_size in list(range(2, 70)) + [100, 127, 128, 1000, 4095, 65537, (1 << 29) + 1, 1 << 30]:
        bits = (page_size - 1).bit_length()
        mul = (1 << (31 + bits)) // page_size + 1
        assert mul < 1 << 32
        top = (1 << 31) - 1
        for key in {0, 1, page_size - 1, page_size, 2 * page_size - 1, top // page_size * page_size - 1, top // page_size * page_size, top}:
            assert (key * mul >> 32) >> (bits - 1) == key // page_size, (key, page_size)
