"""The cache's stored values (4 significant bits, cut to e4m3's grid under a power-of-two scale) on the CPU: the
integer arithmetic that the kernels use against the definition, for every input; and the calls' refusals that need no
device."""
import os
import subprocess

import numpy as np
import pytest

import invariant_tree_ordered_b200 as tbik
from invariant_tree_ordered_b200 import _binding as B
from invariant_tree_ordered_b200 import build as libbuild
from tests import cache_model as cm

HERE = os.path.dirname(os.path.abspath(__file__))
EXPS = [-100, -20, -14, -9, -8, -7, -1, 0, 5, 60, 119, 120]


@pytest.fixture(scope="module")
def tables(tmp_path_factory):
    d = tmp_path_factory.mktemp("cache")
    exe, out = str(d / "check"), str(d / "tables.bin")
    subprocess.check_call([libbuild.nvcc(), "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a", "-I",
                           libbuild.INCLUDE, "-I", libbuild.CSRC, os.path.join(HERE, "cache_math_check.cu"), "-o", exe])
    subprocess.check_call([exe, out])
    raw = open(out, "rb").read()
    n = len(EXPS) * 65536
    quant = np.frombuffer(raw[:n], np.uint8).reshape(len(EXPS), 65536)
    need = np.frombuffer(raw[n:n + 4 * 0x7F80], np.int32)
    down = np.frombuffer(raw[n + 4 * 0x7F80:], np.uint8).reshape(41, 256)
    return quant, need, down


def test_every_bf16_value_under_each_scale(tables):
    h = np.arange(65536)
    x = cm.bf16_to_f64(h)
    for E, got in zip(EXPS, tables[0]):
        r = cm.round4(np.where(np.isfinite(x), x, 0.0))
        ref = cm.cut(r * 2.0 ** -float(E))
        fits = (np.abs(ref) <= 448) & np.isfinite(x)  # larger values cannot meet this scale
        v = cm.E4M3[got]
        assert np.array_equal(v[fits], ref[fits]), E
        assert np.array_equal(np.signbit(v[fits]), np.signbit(x[fits])), E
        inf = np.isinf(x)
        assert np.array_equal(v[inf], np.sign(x[inf]) * 448) and not v[np.isnan(x)].any()


def test_scale_is_the_smallest_that_holds_the_value(tables):
    x = cm.bf16_to_f64(np.arange(0x7F80))
    assert [cm.need(a) for a in cm.round4(x)] == tables[1].tolist()


def test_down_composes_and_matches_the_definition(tables):
    down = tables[2]
    ok = ~np.isnan(cm.E4M3)
    for d in range(41):
        assert np.array_equal(cm.E4M3[down[d]][ok], cm.cut(cm.E4M3[ok] * 2.0 ** -d))
    for a in range(20):
        for b in range(20):  # cutting twice is cutting once: pages do not depend on how tokens arrive
            assert np.array_equal(down[b][down[a]], down[a + b])


def test_quantising_late_equals_quantising_early(tables):
    """A token stored under a small scale and moved down is the token stored under the larger one."""
    quant, _, down = tables
    x = cm.bf16_to_f64(np.arange(65536))
    i, j = EXPS.index(-9), EXPS.index(-7)
    fits = np.isfinite(x) & (np.abs(cm.round4(np.where(np.isfinite(x), x, 0.0))) <= 448 * 2.0 ** -9)
    assert np.array_equal(down[2][quant[i]][fits], quant[j][fits])


def test_host_only_queries_and_refusals():
    lib = tbik.load_library()
    bad = (1 << 64) - 1
    assert lib.tbik_cache_fork_workspace(0) == 8 and lib.tbik_cache_fork_workspace(10) == 88
    assert lib.tbik_cache_fork_workspace(-1) == bad and lib.tbik_cache_fork_workspace(8193) == bad
    assert lib.tbik_cache_compact_workspace(7) == (2 + 8 + 7) * 4
    assert lib.tbik_cache_compact_workspace(0) == bad and lib.tbik_cache_compact_workspace((1 << 20) + 1) == bad
    assert lib.tbik_status_string(B.TBIK_ERR_PAGE) and lib.tbik_status_string(B.TBIK_ERR_VALUE) == b"input is not finite"
    torch = pytest.importorskip("torch")
    table, lens = tbik.cache_table(4, 4, device="cpu")
    pages, scales, refs = tbik.cache_pages(4, 2, 64, 16, device="cpu")
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):  # nothing runs on host tensors
        tbik.cache_extend(table, lens, refs, one, page=16)
    with pytest.raises(TypeError):
        tbik.sample(torch.zeros(1, 8), torch.zeros(1))
    with pytest.raises(TypeError):
        tbik.cache_compact(pages, scales, table, lens, refs)
    with pytest.raises(ValueError):
        tbik.cache_pages(4, 2, 64, 24, device="cpu")


def test_the_position_status_names_packed_offsets():
    """The cache's calls return it for offsets outside the tokens, RoPE for positions outside the table."""
    text = tbik.status_string(B.TBIK_ERR_POSITION)
    assert "RoPE position" in text and "packed token offset" in text and "out of range" in text
