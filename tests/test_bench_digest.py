"""The digest that ties the recorded HBM traffic to the kernels: of the sources of the
workloads' kernels, so that another operator's do not void the record."""
import os
import shutil

import bench


def test_sources():
    names = bench.kernel_sources()
    assert set(bench.WORKLOAD_SOURCES) <= set(names) and {"device_common.h", "gemm_common.h", "gemm_pipe.h"} <= set(names)
    assert not {"kernels.h", "api.cpp", "torch_binding.cpp", "layer_norm.hip", "block_gemm.h"} & set(names)
    assert all(os.path.exists(os.path.join(bench.CSRC, n)) for n in names)


def test_digest_follows_the_workloads_kernels_only(tmp_path):
    csrc = str(tmp_path / "csrc")
    shutil.copytree(bench.CSRC, csrc)
    first = bench.kernel_source_digest(csrc)
    assert first == bench.kernel_source_digest()

    def add(name):
        with open(os.path.join(csrc, name), "a") as f:
            f.write("// more\n")
        return bench.kernel_source_digest(csrc)
    for name in ("layer_norm.hip", "block_gemm.h", "kernels.h", "api.cpp", "another.hip"):
        assert add(name) == first
    for name in ("gemm_mx.hip", "gemm_pipe.h"):
        assert add(name) != first
