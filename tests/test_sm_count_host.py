"""Launch rules ask the device for its number of SMs; the sources name one only as what is
assumed where there is no device."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(__file__), "..", "paged_kv_cache_247_gb300", "csrc")


def test_no_rule_has_a_number_of_sms_of_its_own():
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            for line in f:
                code = line.split("//")[0]
                if re.search(r"\b152\b", code):
                    found.append((os.path.basename(path), code.strip()))
    assert found == [("api.cu", "constexpr int kAssumedSms = 152;")]
