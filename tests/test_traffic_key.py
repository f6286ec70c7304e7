"""The key under which bench.py reports the counter readings of
profiles/traffic.json: it covers every source of the codec's kernels and their
launches, and nothing else."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "lossless_tensor_compression_ibp_amd", "csrc")


def test_sources_are_closed_under_their_includes():
    for name in bench.CODEC_SOURCES:
        with open(os.path.join(CSRC, name)) as f:
            for header in re.findall(r'#include "([a-z_]+\.hpp)"', f.read()):
                assert header in bench.CODEC_SOURCES, (name, header)


def test_key_follows_the_code_of_the_codec_only(tmp_path, monkeypatch):
    csrc = tmp_path / "lossless_tensor_compression_ibp_amd" / "csrc"
    csrc.mkdir(parents=True)
    for name in os.listdir(CSRC):
        if name.endswith((".hip", ".hpp")):
            with open(os.path.join(CSRC, name)) as f:
                (csrc / name).write_text(f.read())
    here = bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() == here
    other = csrc / "ibp_select.hip"
    other.write_text(other.read_text() + "int x;\n")
    commented = csrc / "ibp_decode.hip"
    commented.write_text("// a comment\n" + commented.read_text())
    assert bench.kernel_source_hash() == here
    for name in bench.CODEC_SOURCES:
        text = (csrc / name).read_text()
        (csrc / name).write_text(text + "int x;\n")
        assert bench.kernel_source_hash() != here, name
        (csrc / name).write_text(text)
