"""The paged 4-bit cache at the edges, without a GPU: the workspace's layout, empty batches, the binding's build."""
import os
import subprocess
import sys
import sysconfig

import pytest

from tests.test_paged_host import POS, _append, _attn, _select, dl  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

LAYOUTS = """
#include <cstdio>
#include "paged_layout.h"
int main()
{
    for (int sms = 1; sms <= 400; ++sms)
        for (int D = 64; D <= 128; D += 64)
            for (int QT = 4; QT <= 8; QT += 4) {
                const dlp::AttnLayout l = dlp::attn_layout(sms, D, QT);
                std::printf("%d %d %d %d %zu %zu %zu\\n", sms, D, QT, l.grid, l.counters, l.parts, l.total());
            }
}
"""


def test_workspace_layouts_share_their_counters(tmp_path):
    """On devices of any size the parts of every instance lie behind the counters of all (three a CTA), so that calls of
    different tiles and heads may take turns on one workspace; every part of a CTA has its room."""
    src, exe = tmp_path / "layouts.cpp", tmp_path / "layouts"
    src.write_text(LAYOUTS)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "row_decode_step_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    lines = [[int(x) for x in line.split()] for line in subprocess.check_output([str(exe)], text=True).splitlines()]
    assert len(lines) == 400 * 4
    for sms in range(1, 401):
        mine = [x for x in lines if x[0] == sms]
        most = max(grid * 12 for _, _, _, grid, _, _, _ in mine)
        for _, D, QT, grid, counters, parts, total in mine:
            assert counters >= most and counters % 16 == 0
            assert parts == grid * 2 * QT * (D + 2) * 4 and total == counters + parts


def test_no_rows_need_no_addresses(dl):  # noqa: F811
    """What an empty batch has no elements of may have no address (a torch tensor without elements has none); what it
    has elements of may not."""
    none = dict(q=None, k=None, v=None, pos=None, seq=None, rows=0, qo=None, ko=None, vo=None)
    assert _append(dl, **none) == dl.DL_OK
    assert _append(dl, st=dict(tab=None, seqs=0), **none) == dl.DL_OK
    assert _append(dl, st=dict(tab=None), **none) == dl.DL_E_ARG
    assert _append(dl, st=dict(cs=None), **none) == dl.DL_E_ARG
    none = dict(q=None, out=None, lse=None, rows=0)
    assert _attn(dl, st=dict(tab=None, seqs=0), seqlen=None, **none) == dl.DL_OK
    assert _attn(dl, begin=POS, **none) == dl.DL_OK
    assert _attn(dl, begin=POS, seqlen=None, **none) == dl.DL_E_ARG
    assert _attn(dl, st=dict(tab=None, seqs=0), seqlen=None, begin=POS, rows=3, max_rows=2) == dl.DL_OK
    assert _attn(dl, st=dict(tab=None, seqs=0), seqlen=None, begin=POS, rows=3, q=None) == dl.DL_E_ARG
    assert _attn(dl, st=dict(tab=None, seqs=0), seqlen=None, ws=None, **none) == dl.DL_E_ARG
    assert _attn(dl, st=dict(tab=None, seqs=0), seqlen=None, q=None, out=None, rows=1) == dl.DL_E_ARG
    assert _select(dl, st=dict(tab=None, seqs=0), q=None, seqlen=None, pages=None, rows=0) == dl.DL_OK
    assert _select(dl, st=dict(tab=None, seqs=0), q=None, seqlen=None, pages=None, rows=0, local=0) == dl.DL_E_ARG


def test_build_without_a_host_compiler(dl, monkeypatch, tmp_path):  # noqa: F811
    """Where the binding's compiler (or Python.h) is missing the library is built all the same, with a warning."""
    from row_decode_step_gb300 import _build
    call = tmp_path / os.path.basename(_build.CALL)
    monkeypatch.setattr(_build, "CALL", str(call))
    monkeypatch.setenv("CC", str(tmp_path / "no-such-compiler") + " -pipe")
    with pytest.warns(UserWarning, match="no-such-compiler"):
        assert _build.build() == _build.LIB
    monkeypatch.delenv("CC")
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: paths)
    with pytest.warns(UserWarning, match="Python.h"):
        assert _build.build() == _build.LIB
    assert not call.exists()


def test_binding_is_this_interpreters(dl):  # noqa: F811
    """The binding carries its interpreter's ABI tag, so that another one builds its own; it is the file that is loaded."""
    from row_decode_step_gb300 import _build, paged
    assert os.path.basename(_build.CALL) == "_paged_call" + sysconfig.get_config_var("EXT_SUFFIX")
    assert paged._calls().__file__ == _build.CALL


def test_call_without_the_binding(dl, monkeypatch):  # noqa: F811
    """The paged calls say what is missing where the binding is not built."""
    import row_decode_step_gb300 as pkg
    from row_decode_step_gb300 import paged
    monkeypatch.setattr(paged, "_native", None)
    monkeypatch.delattr(pkg, "_paged_call", raising=False)
    monkeypatch.setitem(sys.modules, "row_decode_step_gb300._paged_call", None)
    with pytest.raises(RuntimeError, match="not built"):
        paged._calls()
