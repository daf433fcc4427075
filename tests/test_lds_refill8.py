"""As tests/test_lds_refill.py, for decoding over a cache in 8 bits (CPU only): an LDS
stage is refilled only after a wait for the reads of it, in the source and in the code
compiled for the GPU.  (Chunks over such a cache, attn8_fwd.hip, go through registers.)"""
import os
import re
import subprocess

import pytest

from tests.test_lds_refill import CSRC, is_tile_copy


@pytest.mark.parametrize("file,refill", [("attn8_decode.hip", "copy_part(b + NS);")])
def test_the_source_waits_before_it_refills(file, refill):
    text = open(os.path.join(CSRC, file)).read()
    at = [m.start() for m in re.finditer(re.escape(refill), text)]
    assert at
    for i in at:
        before = text[:i].rstrip().splitlines()[-3:]
        assert any("wait_lds();" in x or "barrier_lds();" in x for x in before), (file, before)


@pytest.mark.parametrize("file", ["attn8_decode.hip"])
def test_the_compiled_code_waits_before_it_refills(file, tmp_path):
    from chunk_weight_rnn_amd import build
    try:
        cc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = tmp_path / "k.s"
    flags = [f for f in build._flags() if f != "-fPIC"]
    subprocess.run([cc, *flags, "-S", "--offload-device-only", os.path.join(CSRC, file), "-o", str(out)],
                   check=True, capture_output=True)
    copies, reads, early = 0, 0, []
    for n, line in enumerate(out.read_text().splitlines(), 1):
        text = line.split(";")[0].strip()
        if re.match(r"_ZN\S+:", line):
            reads = 0
        elif text and not text.endswith(":") and not text.startswith("."):
            op, _, rest = text.replace("\t", " ").partition(" ")
            rest = rest.strip()
            if op == "ds_read_b128" or op.startswith("ds_read_b64_tr"):
                reads += 1
            elif op == "s_waitcnt" and "lgkmcnt(0)" in rest:
                reads = 0
            elif is_tile_copy(op, rest):
                copies += 1
                if reads:
                    early.append((n, reads))
    assert copies > 0 and not early, early[:5]
