"""What no source of the library may hold (CPU only)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tree_speculative_decoding_masked_gb300", "csrc")


def test_no_bulk_load_is_multicast_over_a_cluster():
    # every copy goes to the shared memory of one CTA, so that replicas of the library on several GPUs of a machine
    # need no multicast objects
    found = []
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r'"\s*"', "", f.read())  # adjacent string literals
        found += [(name, m.group(0)) for m in re.finditer(r"cp\.async\.bulk[\w.:]*multicast[\w:]*", text)]
    assert not found, found
