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
        src.write_text("#include <chrono>\n#include <cstdio>\n#include \"decode.h\"\nint main() {\n  int n; long long v[8];\n"
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


def slices(tokens, groups, warps):
    """Every length of a slice; the longest of equal cost."""
    best = None
    for p in range(groups, 0, -1):
        n = -(-groups // p)
        if n > 1 and tokens * n >= 2 ** 31:
            break
        cost = -(-tokens * n // warps) * (2 * p + 1)
        if best is None or cost < best[0]:
            best = cost, n, p
    return best[1:] if best else (1, 0)


SLICE = "[&] {{ int s, p; mx::rope_slices(v[0], v[1], v[2], &s, &p); return {}; }}()"


def test_slices_of_the_rotation(rule):
    """The least of the busiest warp's cost over all lengths of a slice."""
    args = [(t, g, w) for t in (1, 2, 5, 37, 333, 2432, 4096, 8192, 16384, 100003, 1 << 27, (1 << 31) - 1)
            for g in (*range(0, 40), 72, 100, 257, 1000) for w in (128, 2432, 2560)]
    got = list(zip(rule(SLICE.format("s"), args), rule(SLICE.format("p"), args)))
    for a, x in zip(args, got):
        assert x == slices(*a), a


WATCH = """[&] {
  using clock = std::chrono::steady_clock;
  long long sink = 0;
  const auto t0 = clock::now();
  for (int i = 1; i <= 100; ++i) { int s, p; mx::rope_slices(i, 65535, 2432, &s, &p); sink += s + p; }
  const auto t1 = clock::now();
  for (int i = 1; i <= 100; ++i)
    for (long long p = 65535; p >= 1; --p) sink += (i * ((v[0] + p - 1) / p) + v[1] - 1) / v[1] * (2 * p + 1);
  const auto t2 = clock::now();
  return sink != 0 && (t1 - t0) * 10 < t2 - t1;
}()"""


def test_slices_take_few_steps(rule):
    """The host's time for the most heads: some 500 steps, well below a tenth of that of 65535."""
    assert rule(WATCH, [(65535, 2432)]) == [1]
