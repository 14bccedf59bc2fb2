"""The benchmark's record of the Newton-Schulz launches' DRAM traffic holds for
the sources it was captured on: those of the launches, and no others."""
import os
import shutil

import pytest

import bench

CSRC = os.path.join("matrix_optimizers_zero_gb300", "csrc")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path / CSRC


def edit(path, old, new):
    text = path.read_text(encoding="utf-8")
    assert old in text
    path.write_text(text.replace(old, new, 1), encoding="utf-8")


def test_the_record_is_of_the_present_launches():
    for workload in bench.NS_TRAFFIC:
        assert bench.ns_traffic(workload)[0] is not None


@pytest.mark.parametrize("name,old,new", [
    ("abi.cu", 'return "token index outside the embedding table"', 'return "token outside its table"'),
    ("abi.cu", "int report_cuda(cudaError_t e)", "int report_a_cuda_error(cudaError_t e)"),
    ("embed.cu", "constexpr int kJoin = 32;", "constexpr int kJoin = 16;"),
])
def test_other_sources_leave_the_record(tree, name, old, new):
    edit(tree / name, old, new)
    assert all(bench.ns_traffic(w)[0] is not None for w in bench.NS_TRAFFIC)


@pytest.mark.parametrize("name,old,new", [
    ("abi.cu", "mo::kCounterTilesPerPairLast : mo::kCounterTilesPerPair", "mo::kCounterTilesPerPair : mo::kCounterTilesPerPair"),
    ("abi.cu", "std::min(np.ntiles, dev->sms / 2)", "std::min(np.ntiles, dev->sms / 4)"),
    ("ns_gemm.cu", "namespace mo {", "namespace  mo {"),
    ("mo_internal.h", "kCounterTilesPerPair = 256", "kCounterTilesPerPair = 128"),
    ("plan.cpp", "namespace", "namespace "),
])
def test_the_launches_sources_end_the_record(tree, name, old, new):
    edit(tree / name, old, new)
    assert all(bench.ns_traffic(w)[0] is None for w in bench.NS_TRAFFIC)


def test_a_missing_launch_function_ends_the_record(tree):
    text = (tree / "abi.cu").read_text(encoding="utf-8")
    (tree / "abi.cu").write_text(text.replace("\nint enqueue_muon(", "\nint enqueue_muon_step("), encoding="utf-8")
    assert all(bench.ns_traffic(w)[0] is None for w in bench.NS_TRAFFIC)
