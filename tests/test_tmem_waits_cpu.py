"""TMEM loads write their registers after the instruction: every use has to stand behind a wait
that names them, since nothing else keeps the compiler from moving it in front."""
import os
import re

import pytest

from paged_attention_int8_gb300 import build as pkg_build


def _sources():
    return sorted(f for f in os.listdir(pkg_build.CSRC) if f.endswith((".cu", ".cuh")))


def _text(name):
    with open(os.path.join(pkg_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_one_wait_and_it_names_registers():
    uses = {n: _text(n).count("tcgen05.wait::ld") for n in _sources()}
    assert {n: c for n, c in uses.items() if c} == {"tcgen05.cuh": 1}
    body = _text("tcgen05.cuh").split("tcgen05.wait::ld")[1].split(";\n}")[0]
    assert [int(i) for i in re.findall(r'"\+r"\(r\[(\d+)\]\)', body)] == list(range(32))


@pytest.mark.parametrize("name", [n for n in _sources() if n != "tcgen05.cuh"])
def test_every_load_is_waited_for_by_name(name):
    """The buffers of each run of loads are those of the waits that follow, before anything reads."""
    buffers = lambda call, s: re.findall(call + r"\((?:[^;]*?, )?(\*?[\w:<>()*&\[\] ]+)\);", s)  # noqa: E731
    text = _text(name)
    loads = [b.strip() for b in buffers(r"tc::ld32", text)]
    waits = [b.strip() for b in buffers(r"tc::wait_loaded", text)]
    assert text.count("tc::ld32(") == len(loads) and text.count("tc::wait_loaded(") == len(waits)
    assert loads == waits
