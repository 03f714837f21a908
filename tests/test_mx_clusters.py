"""What the blocks of a cluster tell one another in the kernels of the MXFP4 products
(csrc/mx_product.cu, csrc/mx_pair.cu), without a GPU."""
import os
import re
import subprocess

import pytest

import bit_group_quantized_qgemv_gb300 as q

CSRC = os.path.join(os.path.dirname(q.__file__), "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


# ------------------------------------------------------------------- scopes

@pytest.mark.parametrize("name,shared", [("mx_pair.cu", ("full", "empty", "acc_full", "acc_empty")),
                                         ("mx_product.cu", ("part_full", "part_done"))])
def test_waits_for_other_blocks_are_in_the_clusters_scope(name, shared):
    """Memory is ordered between two blocks by an arrival and a wait that both have the cluster's
    scope; what an arrival or a wait without one (the block's own) orders is undefined there."""
    waits = re.findall(r"step_wait(<true>)?\(smem_u32\(&bars\.(\w+)", source(name))
    assert {bar for _, bar in waits} >= set(shared)
    for scope, bar in waits:
        assert (scope == "<true>") == (bar in shared), f"{name}: {bar}"


def test_arrivals_at_other_blocks_are_in_the_clusters_scope():
    names = [n for n in sorted(os.listdir(CSRC)) if n.endswith((".cu", ".cuh"))]
    found = 0
    for name in names:
        text = source(name)
        for arrive in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text):
            found += 1
            assert ".cluster.shared::cluster" in arrive, f"{name}: {arrive}"
            if ".relaxed." in arrive:                   # (a fence before it, in the same function)
                body = text[:text.index(arrive)].rsplit("__device__", 1)[1]
                assert "fence.release.sync_restrict::shared::cta.cluster" in body, f"{name}: {arrive}"
    assert found > 0
    wait = source("qgemv_device.cuh").split("bool mbar_try_wait_cluster", 1)[1].split("\n}\n", 1)[0]
    assert "relaxed.cluster.shared::cta" in wait
    loop = source("kv_cache.cuh").split("void step_wait(", 1)[1].split("\n}\n", 1)[0]
    assert loop.index("mbar_try_wait_cluster") < loop.index("if (CLUSTER) mbar_acquire_cluster()") < loop.index("__syncwarp")


# ----------------------------------------------------- how many run at a time

def test_numbers_of_clusters(tmp_path):
    exe = str(tmp_path / "clusters")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, os.path.join(here, "clusters_on_cpu.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "done\n", r.stderr


def test_each_kernel_is_asked():
    """A table for each kernel (a template of the kernel, not of its type, which they share)."""
    assert re.search(r"template <auto\* kKernel>\s+int clusters_at_a_time\(", source("mx_product.cuh"))
    pair = source("mx_pair.cu")
    for kernel in ("true, true", "true, false", "false, true", "false, false"):
        assert f"clusters_at_a_time<mx_pair_kernel<{kernel}>>" in pair
    assert "clusters_at_a_time<k>" in source("mx_product.cu")
