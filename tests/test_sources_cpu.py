"""What the sources declare for one another is used."""

import glob
import os
import re

import gqa_attention_learned_gb300 as sa

CSRC = os.path.join(os.path.dirname(sa.__file__), "csrc")


def test_what_files_with_entry_points_share_is_called():
    text = {}
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        with open(path) as f:
            text[os.path.basename(path)] = f.read()
    with open(os.path.join(CSRC, "api.cuh")) as f:
        names = re.findall(r"\b(\w+)\((?:[^()]*)\);", f.read())
    assert "api_status" in names
    for name in names:
        users = [f for f, t in text.items() if f != "sinkattn_api.cu" and re.search(rf"\b{name}\(", t)]
        assert users, f"{name} is declared for other files, and none calls it"
