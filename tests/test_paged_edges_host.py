"""The paged 4-bit cache at the edges, without a GPU: the workspace's layout, empty batches."""
import os
import subprocess

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


def test_no_rows_need_no_addresses(dl):
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
