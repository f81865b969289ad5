"""What the compiler is told about the memory accesses of the gated linear
recurrence (no GPU: device code is only translated)."""
import os
import re
import subprocess

from gated_delta_rule_24_amd import build as B

ACCESS = re.compile(r"(?:load|store) (<\d+ x )?(\w+)>?.*, align (\d+),.*!nontemporal")
BYTES = {"i16": 2, "half": 2, "bfloat": 2, "i32": 4, "float": 4}


def test_vector_accesses_claim_no_alignment(tmp_path):
    """A row of D elements starts on any element where D is no multiple of the vector's length, so no vector
    access may claim more than the smallest element's 2 bytes, and no single element more than its size."""
    out = str(tmp_path / "scan.ll")
    r = subprocess.run([B.HIPCC, *B.COMMON, "--offload-device-only", "-S", "-emit-llvm", "-Xclang",
                        "-disable-llvm-passes", os.path.join(B.CSRC, "gdn_scan.hip"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = [m.groups() for m in map(ACCESS.search, open(out)) if m]
    vectors = [(v + e, int(align)) for v, e, align in found if v]
    assert len(vectors) >= 4 and all(align <= 2 for _, align in vectors), vectors
    assert all(int(align) <= BYTES[e] for v, e, align in found if not v), found
