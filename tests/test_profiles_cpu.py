"""The profiles' digests and the linear layer's summaries: what a digest depends on, and that committed profiles of the
present sources name the kernels that the library plans."""
import csv
import glob
import os
import re
import shutil

import pytest

from bit_quantization_block_amd import linear_workloads as L
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


@pytest.mark.parametrize("name", ["kernels_linear.md", "counters_linear.md"])
def test_linear_profiles_of_the_present_sources_name_the_planned_kernels(name):
    text = open(os.path.join(PROFILES, name)).read()
    if stale(text, "linear"):
        pytest.skip("taken on earlier kernel sources")
    rows = re.findall(r"^\| ([^|]+) \| `([^`]+)` \|", text, flags=re.M)
    assert rows == [(L.label(w), k[0]) for w in L.WORK for k in L.kernels(w)]


def records(passes):
    """What rocprofv3 records of a run, after two kernels that made its inputs and with one of torch's between."""
    out = [("k_mx4_quantize<1, 0>", 16384)] * 2
    for _ in range(passes):
        out += [k for w in L.WORK for k in L.kernels(w)] + [("at::native::other<1>", 7)]
    return out[:-1]


def named(kernel):
    return kernel if kernel.startswith("at::") else f"void lql::(anonymous namespace)::{kernel}(lql::Args, int)"


def test_linear_kernel_summary(tmp_path):
    with open(tmp_path / "t.csv", "w", newline="") as f:
        w = csv.writer(f)
        w.writerow(["Dispatch_Id", "Kernel_Name", "Workgroup_Size_X", "Grid_Size_X", "Grid_Size_Y", "Start_Timestamp", "End_Timestamp"])
        rows = [[i, named(k), 256, 256 * g, 1, 1000 * i, 1000 * i + 100 * (i + 1)] for i, (k, g) in enumerate(records(3))]
        w.writerows(rows[::-1])
    L.summarize_kernels(str(tmp_path / "t.csv"), str(tmp_path / "k.md"), "the command")
    text = (tmp_path / "k.md").read_text()
    order = [(L.label(w), *k) for w in L.WORK for k in L.kernels(w)]
    for j, (label, kernel, groups) in enumerate(order):
        at = [0.1 * (3 + p * (len(order) + 1) + j) for p in range(3)]
        assert f"| {label} | `{kernel}` | {groups} | 3 | {sum(at) / 3:.1f} | {at[0]:.1f} | {at[2]:.1f} |" in text
    assert "`the command`" in text and P.kernel_source_digest("linear") in text


def test_linear_counter_summary(tmp_path):
    files = []
    for i, counters in enumerate(({"SQ_INSTS_VALU": 2e6, "SQ_INSTS_MFMA": 1e6, "SQ_VALU_MFMA_BUSY_CYCLES": 1024 * 500.0},
                                  {"SQ_LDS_IDX_ACTIVE": 256 * 250.0, "SQ_LDS_BANK_CONFLICT": 256 * 25.0, "GRBM_GUI_ACTIVE": 8 * 10000.0},
                                  {"FETCH_SIZE": 5e4}, {"WRITE_SIZE": 3e4})):
        files.append(str(tmp_path / f"{i}.csv"))
        with open(files[-1], "w", newline="") as f:
            w = csv.writer(f)
            w.writerow(["Dispatch_Id", "Kernel_Name", "Workgroup_Size", "Grid_Size", "VGPR_Count", "Counter_Name", "Counter_Value"])
            for d, (k, g) in enumerate(records(2)):
                for name, value in counters.items():
                    w.writerow([d, named(k), 256, 256 * g, 88, name, value])
    L.summarize_counters(str(tmp_path / "c.md"), "the commands", *files)
    text = (tmp_path / "c.md").read_text()
    first = L.WORK[0]
    read, written, _ = L.needed(first)
    assert (f"| {L.label(first)} | `{L.kernels(first)[0][0]}` | 88 | 10000 | 5% | 39% | 2% | 10% | 102 | 31 | "
            f"{read / 1e6:.0f} + {written / 1e6:.0f} |") in text
    assert len(re.findall(r"^\| .* \| `k_", text, flags=re.M)) == sum(len(L.kernels(w)) for w in L.WORK)


def test_a_run_of_other_kernels_is_refused(tmp_path):
    with pytest.raises(SystemExit):
        L._attribute([(k, g, 1.0) for k, g in records(1)][:-1])
