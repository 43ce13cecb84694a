"""CPU checks of include/gemm_decode.h: exports, structs, and refusals that need no GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import tensor_core_gemm_tcgen05_gb300 as g
from tensor_core_gemm_tcgen05_gb300 import _build, decode, serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_decode.h")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return g.lib()


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_exports_match_header(lib):
    funcs = sorted(set(re.findall(r"\b(gemm_\w+)\s*\(", header())))
    assert sorted(g.DECODE_EXPORTS) == funcs
    out = subprocess.run(["nm", "-D", "--defined-only", g.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(funcs) <= exported
    assert int(re.search(r"GEMM_TREE_MAX_WORDS (\d+)", header()).group(1)) == g.GEMM_TREE_MAX_WORDS


def test_structs_match_header(tmp_path):
    structs = {"gemm_tree": decode.Tree, "gemm_kv_seqs": decode.KvSeqs, "gemm_kv_weights": decode.KvWeights, "gemm_w4": decode.W4}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gemm_decode.h"', "int main(void) {"]
    for name, s in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in s._fields_]
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in structs.values():
        want += [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want
    for p, s in zip((decode._TREE, decode._SEQS, decode._WEIGHTS, decode._W4), structs.values()):
        assert p.size == ctypes.sizeof(s)
        values = [i + 1 for i in range(len(s._fields_))]
        x = s.from_buffer_copy(p.pack(*values))
        assert [getattr(x, f[0]) for f in s._fields_] == values


def test_null_arguments_are_rejected(lib):
    h, c, b = (ctypes.byref(s()) for s in (serving.Heads, serving.KvCache, serving.KvBatch))
    t, s, w, w4 = (ctypes.byref(x()) for x in (decode.Tree, decode.KvSeqs, decode.KvWeights, decode.W4))
    assert lib.gemm_tree_mask(None, b, 0, None, None, 1, 1, None, None) == g.GEMM_ERR_ARG
    assert lib.gemm_tree_attention(None, c, b, t, h, 1.0, h, None, 0, None, 0, None) == g.GEMM_ERR_ARG
    assert lib.gemm_tree_attention(None, c, b, None, h, 1.0, h, None, 0, None, 0, None) == g.GEMM_ERR_ARG
    assert lib.gemm_tree_attention_workspace(None, c, b, 8) == g.GEMM_ERR_ARG
    assert lib.gemm_kv_weigh(None, c, b, h, 1.0, None, 0, 0, 1.0, w, None) == g.GEMM_ERR_ARG
    assert lib.gemm_kv_select(None, s, 1, 16, 1, w, 1, 0, 0, None, 1, 1, None, None) == g.GEMM_ERR_ARG
    assert lib.gemm_kv_compact(None, c, s, w, None, 1, 1, 1, None, None, None, None) == g.GEMM_ERR_ARG
    assert lib.gemm_w4_run(None, 0, 1, 8, 32, None, 32, w4, None, None, 8, 0, None) == g.GEMM_ERR_ARG


def test_binding_refuses_what_does_not_fit():
    """Shapes, types and layouts are checked before the library is called (CPU tensors will do)."""
    z = torch.zeros
    q, cache = z(3, 4, 64, dtype=torch.float16), z(5, 2, 16, 64, dtype=torch.float16)
    qs, kv, pt = z(2, dtype=torch.int32), z(1, dtype=torch.int32), z(1, 4, dtype=torch.int32)
    mask, w = z(3, 1, dtype=torch.int32), z(5, 2, 16)
    bad = pytest.raises(ValueError)
    with bad:
        g.tree_mask(None, z(3), qs, kv, 4)
    with bad:
        g.tree_mask(None, z(3, dtype=torch.int32), qs, kv, 2049)
    with bad:
        g.tree_mask(None, z(3, dtype=torch.int32), qs, kv, 4, positions=z(2, dtype=torch.int32))
    for m in (mask[:2], mask.long(), mask[:, 0], z(2, 3, dtype=torch.int32).t()):
        with bad:
            g.tree_attention(None, q, cache, cache.clone(), qs, kv, pt, m)
    for kw in (dict(lse=z(3, 2)), dict(out=q[:2]), dict(workspace=z(4))):
        with bad:
            g.tree_attention(None, q, cache, cache.clone(), qs, kv, pt, mask, **kw)
    for args in ((q.float(), cache, qs, kv, pt, z(3, 4), w), (q, cache, qs, kv, pt, z(3, 3), w), (q, cache, qs, kv, pt, z(3, 4), w[:4]),
                 (q, cache, qs, kv, pt, z(3, 4), w.double()), (q, cache, qs, kv, pt, z(3, 4), z(5, 16, 2).transpose(1, 2)),
                 (q[..., :32], cache, qs, kv, pt, z(3, 4), w), (q, cache[0], qs, kv, pt, z(3, 4), w)):
        with bad:
            g.kv_weigh(None, *args)
    for kw in (dict(keep=-1), dict(keep=4, index=z(1, 2, 3, dtype=torch.int32)), dict(keep=4, counts=z(2, dtype=torch.int32))):
        with bad:
            g.kv_select(None, w, kv, pt, **kw)
    one = z(1, dtype=torch.int32)
    for index, counts, kw in ((z(1, 4), one, {}), (z(2, 4, dtype=torch.int32), one, {}), (z(1, 3, 4, dtype=torch.int32), one, {}),
                              (z(1, 4, dtype=torch.int32), z(2, dtype=torch.int32), {}), (z(1, 4, dtype=torch.int32), one, dict(start=z(1))),
                              (z(1, 4, dtype=torch.int32), one, dict(weights=w[:, :1]))):
        with bad:
            g.kv_compact(None, cache, cache.clone(), kv, pt, index, counts, **kw)
    a, codes, scales, zeros = z(2, 64, dtype=torch.float16), z(8, 32, dtype=torch.uint8), z(8, 2, dtype=torch.float16), z(8, 2, dtype=torch.uint8)
    for args in ((a, codes[:, :31], scales), (a, codes, scales.float()), (a, codes, scales, zeros[:, :1]), (a.t(), codes, scales),
                 (a, codes, scales[:, :0]), (a, codes, z(8, 3, dtype=torch.float16)), (a, codes, scales, zeros, z(7, dtype=torch.float16))):
        with bad:
            g.w4_gemm(None, *args)
