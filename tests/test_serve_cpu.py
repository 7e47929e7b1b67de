"""Host-side checks of the serving entry points (no GPU): struct layouts, workspace sizes, null handles, and the test
helpers themselves."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from approximate_long_context_b200 import binding
from serving import ListCache, attend, tolerances

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from approximate_long_context_b200 import build
    build.build()
    return binding.lib()


@pytest.mark.parametrize("c,py", [("ha_prompt_args", binding.PromptArgs), ("ha_cache", binding.CacheArgs),
                                  ("ha_tree_args", binding.TreeArgs)])
def test_structs_mirror_the_header(tmp_path, c, py):
    fields = [f for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    body = "".join(f'    printf("{f} %zu\\n", offsetof({c}, {f}));\n' for f in fields)
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "hyper_attn.h"\nint main(void) {\n'
                   f'    printf("size %zu\\n", sizeof({c}));\n' + body + "    return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(out["size"]) == ctypes.sizeof(py)
    for f in fields:
        assert int(out[f]) == getattr(py, f).offset, f


@pytest.mark.parametrize("packed,py", [(binding._PROMPT, binding.PromptArgs), (binding._TREE, binding.TreeArgs),
                                       (binding._CACHE, binding.CacheArgs)])
def test_packed_arguments_are_the_struct(packed, py):
    values = list(range(3, 3 + len(py._fields_)))
    raw = packed.pack(*values)
    a = py.from_buffer_copy(raw + bytes(ctypes.sizeof(py) - len(raw)))
    assert [getattr(a, f) for f, _ in py._fields_] == values


def test_null_handles_and_workspaces(lib):
    inv = binding.HA_ERR_INVALID_ARG
    assert lib.hyper_attn_prompt(None, binding.PromptArgs()) == inv
    assert lib.hyper_attn_tree(None, binding.CacheArgs(), binding.TreeArgs()) == inv
    assert lib.hyper_attn_cache_free(None, binding.CacheArgs(), None, 0) == inv
    assert lib.hyper_attn_cache_fork(None, binding.CacheArgs(), None, None, 0) == inv
    assert lib.hyper_attn_cache_reserve(None, binding.CacheArgs(), None, None, 0, None, None, 0) == inv
    assert lib.hyper_attn_cache_append(None, binding.CacheArgs(), None, None, 0, 0, None, None, None, None, 0, 1) == inv
    assert lib.hyper_attn_cache_commit(None, binding.CacheArgs(), None, None, None, 0, 0) == inv
    assert lib.hyper_attn_tree_workspace(None, 64) == 0 and lib.hyper_attn_capturing(None) == 0
    assert lib.hyper_attn_prompt_workspace(None, 1, 1, 1, 1, 1) == 0
    assert lib.hyper_attn_cache_workspace(-1, 5) == 0
    assert lib.hyper_attn_cache_workspace(7, 5) >= 7 * 8


def test_kernel_classes_mirror_the_header():
    text = open(os.path.join(ROOT, "include", "hyper_attn.h")).read()
    for i, name in enumerate(binding.KERNEL_CLASSES):
        assert f"HA_KC_{name.upper()} = {i}," in text
    assert f"HA_KC_COUNT = {len(binding.KERNEL_CLASSES)}" in text


def test_reference_attention_by_hand():
    """Two keys with weights 1/4 and 3/4; a row that sees one key; a row that sees none."""
    q = torch.tensor([1.0, 1.0, 1.0]).view(3, 1, 1)
    k = torch.tensor([0.0, float(np.log(3.0)), float("nan")]).view(3, 1, 1)
    v = torch.tensor([4.0, 8.0, float("nan")]).view(3, 1, 1)
    seen = torch.tensor([[True, True, False], [False, True, False], [False, False, False]])
    o, lse, mag, _ = attend(q, k, v, seen, 1.0)
    assert torch.allclose(o[:2, 0, 0], torch.tensor([7.0, 8.0]).double(), atol=1e-6)
    assert torch.allclose(lse[0, :2], torch.tensor([np.log(4.0), np.log(3.0)]), atol=1e-6) and torch.isneginf(lse[0, 2])
    assert torch.allclose(mag[:2], o[:2].abs())


def test_tolerances_cover_rounded_arithmetic():
    """fp32 arithmetic of the same formula lies within the fp32 tolerance, bf16 weights within theirs and outside the fp32
    one: the bounds are neither too small nor without meaning."""
    g = torch.Generator().manual_seed(0)
    n, d = 200, 64
    q, k, v = (torch.randn(n, 1, d, generator=g) for _ in range(3))
    seen = torch.ones(n, n, dtype=torch.bool).tril()
    want = [x.cpu() for x in attend(q, k, v, seen, 0.125)]
    s = (q[:, 0] @ k[:, 0].T * 0.125).masked_fill(~seen, -float("inf"))
    e = torch.exp(s - s.amax(1, keepdim=True))
    o = (e @ v[:, 0] / e.sum(1, keepdim=True))[:, None]
    ob = (e.bfloat16().float() @ v[:, 0] / e.sum(1, keepdim=True))[:, None]
    tight, _ = tolerances(*want, n, d, out_bf16=False)
    loose, _ = tolerances(*want, n, d, p_bits=2.0 ** -8, out_bf16=False)
    assert ((o.double() - want[0]).abs() <= tight).all()
    assert ((ob.double() - want[0]).abs() <= loose).all() and not ((ob.double() - want[0]).abs() <= tight).all()


def test_list_cache():
    """A shared last page is copied by the first of the two that append to it, the second keeps it."""
    k = np.zeros((1, 8, 1, 4, 2), np.float32)
    c = ListCache(k, k.copy(), 3, 4)
    assert c.reserve([0], [6]) == [6]
    rows = np.arange(12, dtype=np.float32).reshape(1, 6, 1, 2)
    c.append([0], [0, 6], rows, rows)
    c.commit([0], [3], [[0, 2, 5]])
    assert c.lens == [3, 0, 0] and c.rows[0] == [0] and c.refs[:2] == [1, 0]
    assert c.k[0, 0, 0, :3, 0].tolist() == [0, 4, 10]
    c.fork([0], [2])
    assert c.refs[0] == 2
    assert c.reserve([2, 0], [1, 1]) == [1, 1]
    assert c.rows == [[0], [], [1]] and c.refs[:2] == [1, 1]
    assert c.k[0, 1, 0, :3, 0].tolist() == [0, 4, 10]
    assert c.reserve([1, 0], [28, 1]) == [0, 0]        # seven pages, six are free: the first is short, so is all behind it
    c.free([0, 2])
    assert sum(c.refs) == 0
