"""An LDS stage is refilled only after a wait for the reads of it (CPU only).

The attention kernels copy tiles from memory to the LDS by instructions that
write no register, so nothing but a wait keeps a copy behind the reads of what
it overwrites.  Two looks at it: the source has that wait before each refill of
a stage, and in the code compiled for the GPU no copy of a tile follows a
fragment's read without a full wait for LDS accesses between them."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "chunk_weight_rnn_amd", "csrc")


# the loop's refill, and how many waits with LDS accesses in them may stand before it
@pytest.mark.parametrize("file,refill", [("attn_decode.hip", "copy_part(b + 2);"), ("attn_fwd.hip", "copy_tile(j + 1, "),
                                         ("attn_bwd.hip", "copy_tile(j + 1, ")])
def test_the_source_waits_before_it_refills(file, refill):
    text = open(os.path.join(CSRC, file)).read()
    at = [m.start() for m in re.finditer(re.escape(refill), text)]
    assert at
    for i in at:
        before = text[:i].rstrip().splitlines()[-3:]
        assert any("wait_lds();" in x or "barrier_lds();" in x for x in before), (file, before)


@pytest.mark.parametrize("file", ["attn_decode.hip", "attn_fwd.hip", "attn_bwd.hip"])
def test_the_compiled_code_waits_before_it_refills(file, tmp_path):
    from chunk_weight_rnn_amd import build
    try:
        cc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = tmp_path / "k.s"
    flags = [f for f in build._flags() if f != "-fPIC"]
    subprocess.run([cc, *flags, "-S", "--offload-device-only", os.path.join(CSRC, file), "-o", str(out)], check=True,
                   capture_output=True)
    copies, reads, early = 0, 0, []
    for n, line in enumerate(out.read_text().splitlines(), 1):
        s = line.strip()
        if re.match(r"_ZN\S+:", line):
            reads = 0
        elif re.match(r"ds_read_b128|ds_read_b64_tr", s):
            reads += 1
        elif s.startswith("s_waitcnt") and "lgkmcnt(0)" in s:
            reads = 0
        elif s.startswith("global_load_lds_dwordx4") or (s.startswith("buffer_load_dwordx4") and s.endswith(" lds")):
            copies += 1
            if reads:
                early.append((n, reads))
    assert copies > 0 and not early, early[:5]
