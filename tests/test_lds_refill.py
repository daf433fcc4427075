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


@pytest.fixture(scope="module", params=["attn_decode.hip", "attn_fwd.hip", "attn_bwd.hip"])
def code(request, tmp_path_factory):
    """The file's device code: (line number, instruction, operands), None where a function begins."""
    from chunk_weight_rnn_amd import build
    try:
        cc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = tmp_path_factory.mktemp("asm") / "k.s"
    flags = [f for f in build._flags() if f != "-fPIC"]
    subprocess.run([cc, *flags, "-S", "--offload-device-only", os.path.join(CSRC, request.param), "-o", str(out)],
                   check=True, capture_output=True)
    r = []
    for n, line in enumerate(out.read_text().splitlines(), 1):
        text = line.split(";")[0].strip()
        if re.match(r"_ZN\S+:", line):
            r.append(None)
        elif text and not text.endswith(":") and not text.startswith("."):
            op, _, rest = text.partition(" ") if " " in text else text.partition("\t")
            r.append((n, op, rest.strip()))
    return r


def is_tile_copy(op, rest):
    return op == "global_load_lds_dwordx4" or (op == "buffer_load_dwordx4" and rest.endswith(" lds"))


def test_the_compiled_code_waits_before_it_refills(code):
    copies, reads, early = 0, 0, []
    for x in code:
        if x is None:
            reads = 0
            continue
        n, op, rest = x
        if op == "ds_read_b128" or op.startswith("ds_read_b64_tr"):
            reads += 1
        elif op == "s_waitcnt" and "lgkmcnt(0)" in rest:
            reads = 0
        elif is_tile_copy(op, rest):
            copies += 1
            if reads:
                early.append((n, reads))
    assert copies > 0 and not early, early[:5]


def scalars(text):
    r = set()
    for a, b, c in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        r |= {int(c)} if c else set(range(int(a), int(b) + 1))
    return r


def test_resources_of_copies_are_ready(code):
    """A scalar register that a vector instruction wrote (a spilled one that comes
    back among them) may be read by a memory instruction five wait states later at
    the earliest.  The compiler sees to that for its own instructions, not for the
    copies, which are written out."""
    need, copies, early, past = 5, 0, [], []  # past: wait states and scalars written, newest last
    for x in code:
        if x is None:
            past = []
            continue
        n, op, rest = x
        if op == "buffer_load_dwordx4" and rest.endswith(" lds"):
            copies += 1
            reads, states = scalars(rest), 0
            for w, wrote in reversed(past):
                if states >= need:
                    break
                if wrote & reads:
                    early.append((n, states))
                    break
                states += w
        past.append((int(rest) + 1 if op == "s_nop" else 1, scalars(rest.split(",")[0]) if op.startswith("v_") else set()))
        past = past[-need:]
    assert not early, early[:5]
    assert copies > 0
