"""A block must not end while copies into its shared memory are under way: the
memory is the next block's by then.  A kernel whose waits can run out gives up
in any of its roles, also after the loading one has issued its last copy and
looked at the flag; so the loading role waits for its copies whatever the flag
says.  Read from the sources, as the late copy itself must not happen."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_attention_backward_gb300", "csrc")


def code(path):
    text = re.sub(r"//[^\n]*", "", open(path).read())
    return re.sub(r"\s+", " ", text)


@pytest.mark.parametrize("name,full", [("lin_attn.cu", ("Z::kFull", "kOBarFull", "kOBarAFull", "kGBarFull")),
                                       ("forward.cu", ("kFBarKVFull", "kFBarQ")),
                                       ("causal.cu", ("kBarQFull", "kBarDOFull", "kBarKV", "kBarV", "kQBarFull"))])
def test_every_load_is_waited_for(name, full):
    text = code(os.path.join(CSRC, name))
    for bar in full:                                        # a last wait for each barrier that a load completes on
        assert re.search(r"mbar_wait_bounded\(bar\(" + bar + r"\b[^;]*2000000000ull\)", text), bar


def test_no_wait_for_copies_depends_on_who_gave_up():
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = code(path)
        conditions = re.findall(r"if \((\*abort_flag|!ok)\) (\{[^}]*\}|[^;]*;)", text)
        for _, body in conditions:
            assert "mbar_wait_bounded" not in body, (os.path.basename(path), body)
