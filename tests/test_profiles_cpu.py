"""The profiles' digests: what they depend on, and that committed profiles of the present sources name the kernels that
the library plans."""
import glob
import os
import re
import shutil

import pytest

from bit_quantization_block_amd import lq
from bit_quantization_block_amd import profiling as P
from bit_quantization_block_amd import workloads as W

PROFILES = os.path.join(P.ROOT, "profiles")


def test_a_paths_digest_depends_on_its_own_sources(tmp_path):
    """Sources of the linear layer, added or changed, leave the fake-quant kernels' digest, and the other way round."""
    csrc = tmp_path / "bit_quantization_block_amd" / "csrc"
    shutil.copytree(os.path.join(P.ROOT, "bit_quantization_block_amd", "csrc"), csrc)
    shutil.copytree(os.path.join(P.ROOT, "include"), tmp_path / "include")

    def digests():
        return [P.kernel_source_digest(path, str(tmp_path)) for path in ("fake_quant", "linear")]

    def after(path, old, new):
        text = path.read_text()
        assert old in text
        path.write_text(text.replace(old, new, 1))
        return digests()

    here = digests()
    assert here == [P.kernel_source_digest(), P.kernel_source_digest("linear")] and here[0] != here[1]
    fake, linear = here
    header = tmp_path / "include" / "lq.h"
    assert after(header, "LQ_API int lq_mx4_dgrad(", "LQ_API int lq_new(int x);\nLQ_API int lq_mx4_dgrad(") == [fake, linear]
    assert after(header, "  int64_t ld_in; ", "  int64_t ld_new; int64_t ld_in; ")[0] == fake
    assert digests()[1] != linear
    linear = digests()[1]
    for name in P.LINEAR_SOURCES:
        assert after(csrc / name, "namespace", "/* a comment */ namespace") == [fake, linear]
        now = after(csrc / name, "namespace", "int more; namespace")
        assert now[0] == fake and now[1] != linear, name
        linear = now[1]
    for name in ("lq_api.hip", "lq_kernels.h", "lq_fast.h", "lq_lc.hip", "lq_ceiling.hip"):
        now = after(csrc / name, "namespace", "int more; namespace")
        assert now[0] != fake and now[1] == linear, name
        fake = now[0]
    for name in P.SHARED_SOURCES:
        now = after(csrc / name, "namespace", "int more; namespace")
        assert now[0] != fake and now[1] != linear, name
        fake, linear = now
    now = after(header, "  int32_t two_level;", "  int32_t three_level;")
    assert now[0] != fake and now[1] != linear


def stale(text, path):
    m = re.search(r"Kernel source digest: ([0-9a-f]{16})", text)
    return not m or m.group(1) != P.kernel_source_digest(path)


@pytest.mark.parametrize("cfg", sorted(os.path.basename(p)[len("kernels_"):-len(".md")] for p in glob.glob(os.path.join(PROFILES, "kernels_c*.md"))))
def test_profiles_of_the_present_sources_name_the_planned_kernels(cfg):
    text = open(os.path.join(PROFILES, f"kernels_{cfg}.md")).read()
    if stale(text, "fake_quant"):
        pytest.skip("taken on earlier kernel sources")
    listed = set(re.findall(r"\| `([^`]+)` \|", text))
    spec = W.WORKLOADS[cfg]
    for v in spec["variants"]():
        for k in lq.call_kernels(v, spec["dtype"], *spec["shape"]):
            assert k in listed, (cfg, v, k)
