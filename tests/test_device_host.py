"""The question for the device (no GPU): every entry point that launches asks it through one function, so that a device that cannot be
asked and one of another architecture are told apart alike."""

import os
import re

from top_sparse_mla_gb300.build import PKG_DIR

CSRC = os.path.join(PKG_DIR, "csrc")


def test_the_newer_entry_points_share_one_function():
    where = {f: open(os.path.join(CSRC, f)).read() for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh"))}
    defined = [f for f, text in where.items() if re.search(r"^(?:static|inline) int (?:gb300|current)_sms\(", text, re.M)]
    assert defined == ["device.cuh"], defined
    for f in ("dsa_kv8_attn.cu", "dsa_kv8_prefix.cu", "dsa_mla_prefill.cu", "dsa_qk_norm_rope.cu", "dsa_kv_gather.cu"):
        assert "dsa::gb300_sms(&sms)" in where[f], f
