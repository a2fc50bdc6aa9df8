"""The decoding step's rules on sizes, compiled from the header for the host (no GPU)."""
import os
import subprocess

import pytest

from block_scaled_fp4_bf16_gb300 import build as _build

INCLUDE = os.path.join(os.path.dirname(_build.PKG), "include")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """rule(expression of long long arguments v[0], v[1] .., rows of arguments): its values."""
    folder = tmp_path_factory.mktemp("rules")

    def run(expression, rows):
        name = f"rule{abs(hash(expression))}"
        src, exe = folder / f"{name}.cpp", folder / name
        src.write_text("#include <cstdio>\n#include \"decode.h\"\nint main() {\n  int n; long long v[8];\n"
                       "  while (scanf(\"%d\", &n) == 1) {\n    for (int i = 0; i < n; ++i) if (scanf(\"%lld\", &v[i]) != 1) return 1;\n"
                       f"    printf(\"%lld\\n\", static_cast<long long>({expression}));\n  }}\n}}\n")
        subprocess.run(["g++", "-std=c++17", "-O1", "-I", _build.CSRC, "-I", INCLUDE, "-I", os.path.join(CUDA, "include"),
                        str(src), "-o", str(exe)], check=True)
        text = "\n".join(" ".join(map(str, [len(r), *r])) for r in rows)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [int(x) for x in out.split()]
    return run


VOCABS = [1, 4096, 4097, 8192, 16384, 20011, 32000, 32768, 32769, 50257, 131072, 151937, 262144]
ROWS = [1, 2, 9, 10, 18, 19, 37, 38, 64, 76, 77, 152, 153, 256, 304, 305, 1000, 1 << 20]


@pytest.mark.parametrize("most", [8, 16])
@pytest.mark.parametrize("sms", [16, 132, 152])
def test_clusters_of_the_sampling(rule, sms, most):
    """Powers of two up to what the context has room for, each CTA's slice within the kernel's shared memory."""
    args = [(r, v, sms, most) for r in ROWS for v in VOCABS]
    got = rule("mx::sample_ctas(v[0], v[1], v[2], v[3])", args)
    for (r, v, _, _), n in zip(args, got):
        assert n in (1, 2, 4, 8, 16) and n <= most
        assert -(-v // n) <= 262144 // 8
        assert n < 16 or (v > 32768 and r * 16 <= sms)
    assert (16 in got) == (most == 16 and sms >= 16)
