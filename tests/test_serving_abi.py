"""CPU checks of include/gemm_serving.h: exports, constants and structs, the frequency table
against its formulas, and refusals that need no GPU."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import tensor_core_gemm_tcgen05_gb300 as g
from tensor_core_gemm_tcgen05_gb300 import _build, serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_serving.h")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return g.lib()


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_exports_match_header(lib):
    funcs = sorted(set(re.findall(r"\b(gemm_\w+)\s*\(", header())))
    assert sorted(g.SERVING_EXPORTS) == funcs
    out = subprocess.run(["nm", "-D", "--defined-only", g.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(funcs) <= exported


def test_constants_match_header():
    consts = {k: int(v) for k, v in re.findall(r"\b(GEMM_[A-Z_0-9]+)\s*=\s*(-?\d+)", header())}
    assert len(consts) == 6
    for name, value in consts.items():
        assert getattr(g, name) == value, name


def test_structs_match_header(tmp_path):
    """Sizes and field offsets of the binding's structs against the C compiler's."""
    structs = {"gemm_heads": serving.Heads, "gemm_kv_cache": serving.KvCache, "gemm_kv_batch": serving.KvBatch,
               "gemm_rope": serving.Rope}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gemm_serving.h"', "int main(void) {"]
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
    packed = (serving._HEADS, serving._CACHE, serving._BATCH, serving._ROPE)
    assert [p.size for p in packed] == [ctypes.sizeof(s) for s in structs.values()]
    # and field by field: the packed bytes read back through the structs
    for p, s in zip(packed, structs.values()):
        values = [i + 1 for i in range(len(s._fields_))]
        x = s.from_buffer_copy(p.pack(*values))
        assert [getattr(x, f[0]) for f in s._fields_] == values


def turns(table):
    return [(int(w) % 2 ** 64) / 2 ** 64 for w in table.tolist()]


@pytest.mark.parametrize("rd", [16, 48, 128])
@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
def test_rope_table_matches_formulas(lib, rd, scaling):
    base, factor, original = 10000.0, 8.0, 4096
    table, scale = g.rope_table(rd, base, scaling, factor, original)
    assert table.dtype == torch.int64 and table.shape == (rd // 2,)
    for i, got in enumerate(turns(table)):
        f = base ** (-2 * i / rd)
        if scaling == "linear":
            f = f / factor
        elif scaling == "ntk":
            f = (base * factor ** (rd / (rd - 2))) ** (-2 * i / rd)
        elif scaling == "yarn":
            r = original * f / (2 * math.pi)
            mix = min(1.0, max(0.0, (r - 1) / 31))
            f = (1 - mix) * f / factor + mix * f
        # a few roundings of 2^-53 each, then to a unit of 2^-64
        assert abs(got - f / (2 * math.pi)) <= 1e-14 * f + 2.0 ** -64
    assert scale == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0, rel=1e-6)


def test_rope_table_refusals(lib):
    for kw in (dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=0), dict(base=1.0), dict(base=math.nan),
               dict(base=math.inf), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.inf),
               dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original=-1)):
        with pytest.raises(g.GemmError) as e:
            g.rope_table(**{"rotary_dim": 64, **kw})
        assert e.value.status == g.GEMM_ERR_ARG, kw
    with pytest.raises(ValueError):
        g.rope_table(64, scaling="other")
    assert lib.gemm_rope_table(64, 10000.0, 0, 1.0, 0.0, None, None) == g.GEMM_ERR_ARG
    assert lib.gemm_rope_table(64, 10000.0, 4, 1.0, 0.0, torch.empty(32, dtype=torch.int64).data_ptr(), None) == g.GEMM_ERR_ARG


def test_null_arguments_are_rejected(lib):
    h, c, b, r = (ctypes.byref(s()) for s in (serving.Heads, serving.KvCache, serving.KvBatch, serving.Rope))
    assert lib.gemm_qk_rope(None, 0, 1, 128, h, h, None, r, h, h, None) == g.GEMM_ERR_ARG
    assert lib.gemm_kv_append(None, c, b, h, h, h, r, h, None) == g.GEMM_ERR_ARG
    assert lib.gemm_paged_attention(None, c, b, h, 1.0, h, None, 0, None, 0, None) == g.GEMM_ERR_ARG
    assert lib.gemm_paged_attention_workspace(None, c, b, 8) == g.GEMM_ERR_ARG
    assert g.gemm_status_string(g.GEMM_ERR_INDEX).startswith("GEMM_ERR_INDEX")


def test_binding_refuses_what_does_not_fit():
    """Shapes, types and layouts are checked before the library is called (CPU tensors will do)."""
    z = torch.zeros
    q, k = z(3, 4, 64, dtype=torch.float16), z(3, 2, 64, dtype=torch.float16)
    cache = z(5, 2, 16, 64, dtype=torch.float16)
    qs, kv, pt = z(2, dtype=torch.int32), z(1, dtype=torch.int32), z(1, 4, dtype=torch.int32)
    pos = z(3, dtype=torch.int32)
    for args in ((q.float(), k, pos), (q, k.bfloat16(), pos), (q, k[:2], pos), (q, k, pos.long()), (q, k, pos[:2]),
                 (q.transpose(1, 2), k, pos), (q[0], k, pos)):
        with pytest.raises(ValueError):
            g.qk_rope(None, *args)
    with pytest.raises(ValueError):
        g.qk_rope(None, q, k, pos, q_out=z(3, 4, 128, dtype=torch.float16))
    with pytest.raises(ValueError):
        g.qk_rope(None, q, k, pos, z(16, dtype=torch.int32))
    with pytest.raises(ValueError):
        g.qk_rope(None, q, k, pos, q_norm=z(64))
    for args in ((q, k, k, cache, cache[:4], qs, kv, pt), (q, k, k, cache, cache, qs, kv[:0], pt), (q, k, k[:, :1], cache, cache, qs, kv, pt),
                 (q, z(3, 3, 64, dtype=torch.float16), z(3, 3, 64, dtype=torch.float16), cache, cache, qs, kv, pt),
                 (q, k, k, cache, cache, qs, kv, pt[0]), (q, k, k, cache, cache, qs, kv, pt.t().contiguous().t().expand(1, 4)[:, ::2])):
        with pytest.raises(ValueError):
            g.kv_append(None, *args)
    with pytest.raises(ValueError):
        g.kv_append(None, q, k, k, cache, cache, qs, kv, pt, prefix_len=8)
    for kw in (dict(lse=z(3, 2)), dict(lse=z(3, 4, dtype=torch.float16)), dict(out=q[:2]), dict(workspace=z(4))):
        with pytest.raises(ValueError):
            g.paged_attention(None, q, cache, cache, qs, kv, pt, **kw)
